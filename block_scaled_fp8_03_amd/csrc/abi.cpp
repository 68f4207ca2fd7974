// abi.cpp -- the C entry points declared in include/fp8bs.h.  Each one checks
// its arguments on the host (no HIP call happens before the checks pass) and
// then enqueues the kernels on the caller's stream.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fp8bs.h"
#include "launch.h"

namespace {

// The tile kernels address operands with 32-bit byte offsets and may touch up
// to 256 rows past the end of an operand (those loads return zeros), so
// (rows + 256) * K must stay below 2^32 for A and for (each expert's) B.
constexpr int64_t kLimit32 = (int64_t)1 << 32;
constexpr int64_t kLimitInt = ((int64_t)1 << 31) - 1;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// [p, p + n) and [q, q + m) intersect (empty ranges never do)
bool overlap(const void* p, int64_t n, const void* q, int64_t m) {
  if (n <= 0 || m <= 0) return false;
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

// product of non-negative sizes, or -1 on int64 overflow
int64_t mul(int64_t a, int64_t b) {
  if (a == 0 || b == 0) return 0;
  if (a > INT64_MAX / b) return -1;
  return a * b;
}

int status_of(hipError_t e) { return e == hipSuccess ? FP8BS_OK : FP8BS_ERR_HIP; }

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

extern "C" {

const char* fp8bs_status_string(int status) {
  switch (status) {
    case FP8BS_OK: return "ok";
    case FP8BS_ERR_NULL: return "a required pointer is NULL";
    case FP8BS_ERR_SHAPE: return "invalid shape (negative size, K not a multiple of 128, or size limit exceeded)";
    case FP8BS_ERR_ALIGN: return "a pointer is not aligned as required (16 bytes for tensors, 4 for scales)";
    case FP8BS_ERR_ENUM: return "unknown scale_fmt or out_dtype";
    case FP8BS_ERR_HIP: return "HIP kernel launch failed";
    case FP8BS_ERR_ALIAS: return "an output buffer overlaps an input buffer";
    default: return "unknown status";
  }
}

int fp8bs_version(void) { return 10000; }

int fp8bs_act_quant(const void* x_bf16, void* q_e4m3, float* s, int64_t M, int64_t K,
                    int scale_fmt, void* stream) {
  if (M < 0 || K < 0 || K % 128 != 0) return FP8BS_ERR_SHAPE;
  if (scale_fmt != FP8BS_SCALE_FP32 && scale_fmt != FP8BS_SCALE_UE8M0) return FP8BS_ERR_ENUM;
  const int64_t n = mul(M, K);
  if (n < 0 || mul(n, 2) < 0 || !fp8bs::act_quant_fits(M, K)) return FP8BS_ERR_SHAPE;
  if (n == 0) return FP8BS_OK;
  if (!x_bf16 || !q_e4m3 || !s) return FP8BS_ERR_NULL;
  if (!aligned(x_bf16, 16) || !aligned(q_e4m3, 16) || !aligned(s, 4)) return FP8BS_ERR_ALIGN;
  const int64_t ns = n / 128;
  if (overlap(q_e4m3, n, x_bf16, 2 * n) || overlap(s, 4 * ns, x_bf16, 2 * n) ||
      overlap(q_e4m3, n, s, 4 * ns))
    return FP8BS_ERR_ALIAS;
  return status_of(fp8bs::launch_act_quant(x_bf16, q_e4m3, s, M, K,
                                           scale_fmt == FP8BS_SCALE_UE8M0, (hipStream_t)stream));
}

int fp8bs_e4m3_encode(const float* x, void* q_e4m3, int64_t n, void* stream) {
  if (n < 0 || !fp8bs::e4m3_encode_fits(n)) return FP8BS_ERR_SHAPE;
  if (n == 0) return FP8BS_OK;
  if (!x || !q_e4m3) return FP8BS_ERR_NULL;
  if (!aligned(x, 16) || !aligned(q_e4m3, 4)) return FP8BS_ERR_ALIGN;
  if (overlap(q_e4m3, n, x, 4 * n)) return FP8BS_ERR_ALIAS;
  return status_of(fp8bs::launch_e4m3_encode(x, q_e4m3, n, (hipStream_t)stream));
}

static int weight_quant_entry(bool ue8m0, const void* w_bf16, void* q_e4m3, float* s, int64_t N,
                              int64_t K, void* stream) {
  if (N < 0 || K < 0) return FP8BS_ERR_SHAPE;
  const int64_t n = mul(N, K);
  if (n < 0 || mul(n, 2) < 0 || cdiv(N, 128) > 65535 || cdiv(K, 128) > kLimitInt)
    return FP8BS_ERR_SHAPE;
  if (n == 0) return FP8BS_OK;
  if (!w_bf16 || !q_e4m3 || !s) return FP8BS_ERR_NULL;
  if (!aligned(w_bf16, 16) || !aligned(q_e4m3, 16) || !aligned(s, 4)) return FP8BS_ERR_ALIGN;
  const int64_t ns = cdiv(N, 128) * cdiv(K, 128);
  if (overlap(q_e4m3, n, w_bf16, 2 * n) || overlap(s, 4 * ns, w_bf16, 2 * n) ||
      overlap(q_e4m3, n, s, 4 * ns))
    return FP8BS_ERR_ALIAS;
  return status_of(fp8bs::launch_weight_quant(w_bf16, q_e4m3, s, N, K, ue8m0, (hipStream_t)stream));
}

int fp8bs_weight_quant(const void* w_bf16, void* q_e4m3, float* s, int64_t N, int64_t K,
                       void* stream) {
  return weight_quant_entry(false, w_bf16, q_e4m3, s, N, K, stream);
}

int fp8bs_weight_quant_ue8m0(const void* w_bf16, void* q_e4m3, float* s, int64_t N, int64_t K,
                             void* stream) {
  return weight_quant_entry(true, w_bf16, q_e4m3, s, N, K, stream);
}

int fp8bs_weight_dequant(const void* w_e4m3, const float* s, void* y_bf16, int64_t N, int64_t K,
                         void* stream) {
  if (N < 0 || K < 0) return FP8BS_ERR_SHAPE;
  const int64_t n = mul(N, K);
  if (n < 0 || mul(n, 2) < 0 || !fp8bs::weight_dequant_fits(N, K)) return FP8BS_ERR_SHAPE;
  if (n == 0) return FP8BS_OK;
  if (!w_e4m3 || !s || !y_bf16) return FP8BS_ERR_NULL;
  if (!aligned(w_e4m3, 16) || !aligned(y_bf16, 16) || !aligned(s, 4)) return FP8BS_ERR_ALIGN;
  const int64_t ns = cdiv(N, 128) * cdiv(K, 128);
  if (overlap(y_bf16, 2 * n, w_e4m3, n) || overlap(y_bf16, 2 * n, s, 4 * ns)) return FP8BS_ERR_ALIAS;
  return status_of(fp8bs::launch_weight_dequant(w_e4m3, s, y_bf16, N, K, (hipStream_t)stream));
}

static int gemm_entry(bool ue8m0, const void* a, const float* a_s, const void* b, const float* b_s,
                      void* c, int64_t M, int64_t N, int64_t K, int out_dtype, void* stream) {
  if (M < 0 || N < 0 || K < 128 || K % 128 != 0) return FP8BS_ERR_SHAPE;
  if (out_dtype != FP8BS_OUT_BF16 && out_dtype != FP8BS_OUT_F32) return FP8BS_ERR_ENUM;
  if (M > kLimitInt || N > kLimitInt || K > kLimitInt) return FP8BS_ERR_SHAPE;
  const int64_t na = mul(M, K), nb = mul(N, K), nc = mul(M, N);
  if (na < 0 || nb < 0 || nc < 0 || mul(M + 256, K) >= kLimit32 || mul(N + 256, K) >= kLimit32 ||
      mul(nc, 4) < 0)
    return FP8BS_ERR_SHAPE;
  if (nc == 0) return FP8BS_OK;
  if (!a || !a_s || !b || !b_s || !c) return FP8BS_ERR_NULL;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(c, 16) || !aligned(a_s, 4) ||
      !aligned(b_s, 4))
    return FP8BS_ERR_ALIGN;
  const int64_t cb = nc * (out_dtype == FP8BS_OUT_F32 ? 4 : 2);
  const int64_t nas = M * (K / 128) * 4, nbs = cdiv(N, 128) * (K / 128) * 4;
  if (overlap(c, cb, a, na) || overlap(c, cb, b, nb) || overlap(c, cb, a_s, nas) ||
      overlap(c, cb, b_s, nbs))
    return FP8BS_ERR_ALIAS;
  const bool f32 = out_dtype == FP8BS_OUT_F32;
  return status_of(ue8m0 ? fp8bs::launch_gemm_ue8m0(a, a_s, b, b_s, c, M, N, K, f32, (hipStream_t)stream)
                         : fp8bs::launch_gemm(a, a_s, b, b_s, c, M, N, K, f32, (hipStream_t)stream));
}

int fp8bs_gemm(const void* a, const float* a_s, const void* b, const float* b_s, void* c,
               int64_t M, int64_t N, int64_t K, int out_dtype, void* stream) {
  return gemm_entry(false, a, a_s, b, b_s, c, M, N, K, out_dtype, stream);
}

int fp8bs_gemm_ue8m0(const void* a, const float* a_s, const void* b, const float* b_s, void* c,
                     int64_t M, int64_t N, int64_t K, int out_dtype, void* stream) {
  return gemm_entry(true, a, a_s, b, b_s, c, M, N, K, out_dtype, stream);
}

int fp8bs_moe_gemm(const void* a, const float* a_s, const void* b, const float* b_s,
                   const int32_t* offsets, void* c, int64_t R, int64_t E, int64_t N, int64_t K,
                   int out_dtype, void* stream) {
  if (R < 0 || E < 0 || N < 0 || K < 128 || K % 128 != 0) return FP8BS_ERR_SHAPE;
  if (out_dtype != FP8BS_OUT_BF16 && out_dtype != FP8BS_OUT_F32) return FP8BS_ERR_ENUM;
  if (R > kLimitInt || E > kLimitInt || N > kLimitInt || K > kLimitInt) return FP8BS_ERR_SHAPE;
  const int64_t na = mul(R, K), nbe = mul(N, K), nb = mul(E, nbe), nc = mul(R, N);
  if (na < 0 || nbe < 0 || nb < 0 || nc < 0 || mul(R + 256, K) >= kLimit32 ||
      mul(N + 256, K) >= kLimit32 || mul(nc, 4) < 0)
    return FP8BS_ERR_SHAPE;
  // the launch grid is at most (R / 256 + 2 E) * ceil(N / 256) + 16 workgroups
  if (mul(R / 64 + 2 * E, cdiv(N, 256)) > kLimitInt - 16) return FP8BS_ERR_SHAPE;
  if (nc == 0 || E == 0) return FP8BS_OK;
  if (!a || !a_s || !b || !b_s || !offsets || !c) return FP8BS_ERR_NULL;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(c, 16) || !aligned(a_s, 4) ||
      !aligned(b_s, 4) || !aligned(offsets, 4))
    return FP8BS_ERR_ALIGN;
  const int64_t cb = nc * (out_dtype == FP8BS_OUT_F32 ? 4 : 2);
  const int64_t nas = R * (K / 128) * 4, nbs = E * cdiv(N, 128) * (K / 128) * 4;
  if (overlap(c, cb, a, na) || overlap(c, cb, b, nb) || overlap(c, cb, a_s, nas) ||
      overlap(c, cb, b_s, nbs) || overlap(c, cb, offsets, 4 * (E + 1)))
    return FP8BS_ERR_ALIAS;
  return status_of(fp8bs::launch_moe_gemm(a, a_s, b, b_s, offsets, c, R, E, N, K,
                                          out_dtype == FP8BS_OUT_F32, (hipStream_t)stream));
}

int fp8bs_w8a16_gemm(const void* x_bf16, const void* w_e4m3, const float* w_s, void* c, int64_t M,
                     int64_t N, int64_t K, int out_dtype, void* stream) {
  if (M < 0 || N < 0 || K < 128 || K % 128 != 0) return FP8BS_ERR_SHAPE;
  if (out_dtype != FP8BS_OUT_BF16 && out_dtype != FP8BS_OUT_F32) return FP8BS_ERR_ENUM;
  if (M > kLimitInt || N > kLimitInt || K > kLimitInt) return FP8BS_ERR_SHAPE;
  const int64_t nx = mul(M, K), nw = mul(N, K), nc = mul(M, N);
  if (nx < 0 || nw < 0 || nc < 0 || mul(M + 256, 2 * K) >= kLimit32 || mul(N + 256, K) >= kLimit32 ||
      mul(nc, 4) < 0 || mul(cdiv(M, 256), cdiv(N, 256)) > kLimitInt)
    return FP8BS_ERR_SHAPE;
  if (nc == 0) return FP8BS_OK;
  if (!x_bf16 || !w_e4m3 || !w_s || !c) return FP8BS_ERR_NULL;
  if (!aligned(x_bf16, 16) || !aligned(w_e4m3, 16) || !aligned(c, 16) || !aligned(w_s, 4))
    return FP8BS_ERR_ALIGN;
  const int64_t cb = nc * (out_dtype == FP8BS_OUT_F32 ? 4 : 2);
  const int64_t nws = cdiv(N, 128) * (K / 128) * 4;
  if (overlap(c, cb, x_bf16, 2 * nx) || overlap(c, cb, w_e4m3, nw) || overlap(c, cb, w_s, nws))
    return FP8BS_ERR_ALIAS;
  return status_of(fp8bs::launch_w8a16_gemm(x_bf16, w_e4m3, w_s, c, M, N, K,
                                            out_dtype == FP8BS_OUT_F32, (hipStream_t)stream));
}

static int mla_entry(bool value_side, const void* in, int64_t ld_t, int64_t ld_h, const void* w,
                     const float* w_s, void* out, int64_t T, int64_t H, int64_t dn, int64_t dv,
                     int64_t R, int out_dtype, void* stream) {
  if (T < 0 || H < 0 || ld_t < 0 || ld_h < 0 || dn <= 0 || dv <= 0 || R <= 0 || dn % 128 != 0 ||
      dv % 128 != 0 || R % 128 != 0)
    return FP8BS_ERR_SHAPE;
  if (value_side ? R > 512 : (dn != 128 && dn != 256)) return FP8BS_ERR_SHAPE;
  if (out_dtype != FP8BS_OUT_BF16 && out_dtype != FP8BS_OUT_F32) return FP8BS_ERR_ENUM;
  if (ld_t % 8 != 0 || ld_h % 8 != 0) return FP8BS_ERR_ALIGN;
  const int64_t width = value_side ? R : dn, ncol = value_side ? dv : R;
  const int64_t nrows = mul(H, dn + dv), nw = mul(nrows, R), nout = mul(mul(T, H), ncol);
  // every element offset the kernels form fits an int
  if (nrows < 0 || nw < 0 || nout < 0 || nw > kLimitInt || nout > kLimitInt || ld_t > kLimitInt ||
      ld_h > kLimitInt || dn + dv > kLimitInt)
    return FP8BS_ERR_SHAPE;
  if (nout == 0) return FP8BS_OK;
  const int64_t nin = mul(T - 1, ld_t) + mul(H - 1, ld_h) + width;   // input extent (elements)
  if (nin > kLimitInt || mul(H, cdiv(T, 256)) > kLimitInt) return FP8BS_ERR_SHAPE;
  if (!in || !w || !w_s || !out) return FP8BS_ERR_NULL;
  if (!aligned(in, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(w_s, 4))
    return FP8BS_ERR_ALIGN;
  const int64_t ob = nout * (out_dtype == FP8BS_OUT_F32 ? 4 : 2);
  const int64_t nws = (nrows / 128) * (R / 128) * 4;
  if (overlap(out, ob, in, 2 * nin) || overlap(out, ob, w, nw) || overlap(out, ob, w_s, nws))
    return FP8BS_ERR_ALIAS;
  const bool f32 = out_dtype == FP8BS_OUT_F32;
  return status_of(value_side
                       ? fp8bs::launch_mla_absorb_value(in, ld_t, ld_h, w, w_s, out, T, H, dn, dv,
                                                        R, f32, (hipStream_t)stream)
                       : fp8bs::launch_mla_absorb_key(in, ld_t, ld_h, w, w_s, out, T, H, dn, dv, R,
                                                      f32, (hipStream_t)stream));
}

int fp8bs_mla_absorb_key(const void* q_bf16, int64_t ld_t, int64_t ld_h, const void* wkv_b,
                         const float* wkv_b_s, void* out, int64_t T, int64_t H, int64_t dn,
                         int64_t dv, int64_t R, int out_dtype, void* stream) {
  return mla_entry(false, q_bf16, ld_t, ld_h, wkv_b, wkv_b_s, out, T, H, dn, dv, R, out_dtype,
                   stream);
}

int fp8bs_mla_absorb_value(const void* x_bf16, int64_t ld_t, int64_t ld_h, const void* wkv_b,
                           const float* wkv_b_s, void* out, int64_t T, int64_t H, int64_t dn,
                           int64_t dv, int64_t R, int out_dtype, void* stream) {
  return mla_entry(true, x_bf16, ld_t, ld_h, wkv_b, wkv_b_s, out, T, H, dn, dv, R, out_dtype,
                   stream);
}

int64_t fp8bs_moe_route_workspace_size(int64_t T, int64_t topk, int64_t E) {
  if (T < 0 || topk < 1 || E < 1 || E > kLimitInt) return -1;
  const int64_t P = mul(T, topk);
  if (P < 0 || P > kLimitInt) return -1;
  const int64_t bytes = mul(mul(cdiv(P, 512), E), 4);
  return bytes < 0 ? -1 : bytes;
}

int fp8bs_moe_route(const int32_t* indices, int64_t T, int64_t topk, int64_t E, int32_t* offsets,
                    int32_t* row_token, int32_t* row_of, void* workspace,
                    int64_t workspace_bytes, void* stream) {
  const int64_t need = fp8bs_moe_route_workspace_size(T, topk, E);
  if (need < 0) return FP8BS_ERR_SHAPE;
  if (workspace_bytes < need) return FP8BS_ERR_SHAPE;
  const int64_t P = T * topk;
  if (!offsets) return FP8BS_ERR_NULL;
  if (P > 0 && (!indices || !row_token || !row_of || !workspace)) return FP8BS_ERR_NULL;
  if (!aligned(indices, 4) || !aligned(offsets, 4) || !aligned(row_token, 4) ||
      !aligned(row_of, 4) || !aligned(workspace, 4))
    return FP8BS_ERR_ALIGN;
  const int64_t ob = 4 * (E + 1), pb = 4 * P;
  if (overlap(offsets, ob, indices, pb) || overlap(row_token, pb, indices, pb) ||
      overlap(row_of, pb, indices, pb) || overlap(offsets, ob, row_token, pb) ||
      overlap(offsets, ob, row_of, pb) || overlap(row_token, pb, row_of, pb) ||
      overlap(workspace, need, indices, pb) || overlap(workspace, need, offsets, ob) ||
      overlap(workspace, need, row_token, pb) || overlap(workspace, need, row_of, pb))
    return FP8BS_ERR_ALIAS;
  return status_of(fp8bs::launch_moe_route(indices, T, topk, E, offsets, row_token, row_of,
                                           workspace, (hipStream_t)stream));
}

int fp8bs_moe_route_noalloc(const int32_t* indices, int64_t T, int64_t topk, int64_t E,
                            int32_t* offsets, int32_t* row_token, int32_t* row_of, void* stream) {
  const int64_t need = fp8bs_moe_route_workspace_size(T, topk, E);
  if (need < 0 || need > fp8bs::kRouteScratchBytes) return FP8BS_ERR_SHAPE;
  const int64_t P = T * topk;
  if (!offsets) return FP8BS_ERR_NULL;
  if (P > 0 && (!indices || !row_token || !row_of)) return FP8BS_ERR_NULL;
  if (!aligned(indices, 4) || !aligned(offsets, 4) || !aligned(row_token, 4) || !aligned(row_of, 4))
    return FP8BS_ERR_ALIGN;
  const int64_t ob = 4 * (E + 1), pb = 4 * P;
  if (overlap(offsets, ob, indices, pb) || overlap(row_token, pb, indices, pb) ||
      overlap(row_of, pb, indices, pb) || overlap(offsets, ob, row_token, pb) ||
      overlap(offsets, ob, row_of, pb) || overlap(row_token, pb, row_of, pb))
    return FP8BS_ERR_ALIAS;
  return status_of(fp8bs::launch_moe_route_noalloc(indices, T, topk, E, offsets, row_token, row_of,
                                                   (hipStream_t)stream));
}

int fp8bs_moe_quant_scatter(const void* x_bf16, const int32_t* row_of, void* q_e4m3, float* s,
                            int64_t T, int64_t topk, int64_t R, int64_t K, int scale_fmt,
                            void* stream) {
  if (T < 0 || topk < 1 || R < 0 || K < 0 || K % 128 != 0) return FP8BS_ERR_SHAPE;
  if (scale_fmt != FP8BS_SCALE_FP32 && scale_fmt != FP8BS_SCALE_UE8M0) return FP8BS_ERR_ENUM;
  const int64_t nx = mul(T, K), nq = mul(R, K), P = mul(T, topk);
  if (nx < 0 || nq < 0 || P < 0 || P > kLimitInt || mul(nx, 2) < 0 || R > kLimitInt ||
      !fp8bs::act_quant_fits(T, K))
    return FP8BS_ERR_SHAPE;
  if (nx == 0 || nq == 0) return FP8BS_OK;
  if (!x_bf16 || !row_of || !q_e4m3 || !s) return FP8BS_ERR_NULL;
  if (!aligned(x_bf16, 16) || !aligned(q_e4m3, 16) || !aligned(s, 4) || !aligned(row_of, 4))
    return FP8BS_ERR_ALIGN;
  const int64_t ns = 4 * (nq / 128);
  if (overlap(q_e4m3, nq, x_bf16, 2 * nx) || overlap(s, ns, x_bf16, 2 * nx) ||
      overlap(q_e4m3, nq, s, ns) || overlap(q_e4m3, nq, row_of, 4 * P) ||
      overlap(s, ns, row_of, 4 * P))
    return FP8BS_ERR_ALIAS;
  return status_of(fp8bs::launch_moe_quant_scatter(x_bf16, row_of, q_e4m3, s, T, topk, R, K,
                                                   scale_fmt == FP8BS_SCALE_UE8M0,
                                                   (hipStream_t)stream));
}

int fp8bs_moe_combine(const void* out_bf16, const float* w, const int32_t* row_of, void* y,
                      int64_t T, int64_t topk, int64_t R, int64_t N, int out_dtype, void* stream) {
  if (T < 0 || topk < 1 || R < 0 || N < 0) return FP8BS_ERR_SHAPE;
  if (out_dtype != FP8BS_OUT_BF16 && out_dtype != FP8BS_OUT_F32) return FP8BS_ERR_ENUM;
  const int64_t no = mul(R, N), ny = mul(T, N), P = mul(T, topk);
  if (no < 0 || ny < 0 || P < 0 || P > kLimitInt || mul(no, 2) < 0 || mul(ny, 4) < 0 ||
      R > kLimitInt)
    return FP8BS_ERR_SHAPE;
  if (ny == 0) return FP8BS_OK;
  if (!w || !row_of || !y || (no > 0 && !out_bf16)) return FP8BS_ERR_NULL;
  if (!aligned(out_bf16, 16) || !aligned(y, 16) || !aligned(w, 4) || !aligned(row_of, 4))
    return FP8BS_ERR_ALIGN;
  const int64_t yb = ny * (out_dtype == FP8BS_OUT_F32 ? 4 : 2);
  if (overlap(y, yb, out_bf16, 2 * no) || overlap(y, yb, w, 4 * P) || overlap(y, yb, row_of, 4 * P))
    return FP8BS_ERR_ALIAS;
  return status_of(fp8bs::launch_moe_combine(out_bf16, w, row_of, y, T, topk, R, N,
                                             out_dtype == FP8BS_OUT_F32, (hipStream_t)stream));
}

// rows that a launch has a workgroup of 256 threads for (it has at most 2^32 - 1 threads)
static const int64_t kLimitRows = (1 << 24) - 1;

// columns of a page table, and sequences (the search for a token's looks up to 64 boundaries past them)
static const int64_t kLimitPages = 1 << 30, kLimitSeqs = 1 << 30;

// what the paged-cache entry points share: sizes, format, pointers and alignment of the cache
static int cache_checks(const void* latent, const float* lat_scale, const void* rope, int cache_fmt,
                        int64_t B, int64_t W, int64_t P, int64_t ps, int64_t R, int64_t dr) {
  if (R != 512 || dr != 64 || B < 0 || B > kLimitInt || W < 1 || W > kLimitPages || P < 1 || ps < 1 || ps > 4096 || P > kLimitInt / ps ||
      mul(B, W) < 0 || mul(mul(B, W), 4) < 0)
    return FP8BS_ERR_SHAPE;
  if (cache_fmt != FP8BS_CACHE_BF16 && cache_fmt != FP8BS_CACHE_FP8) return FP8BS_ERR_ENUM;
  if (!latent || !rope || (cache_fmt == FP8BS_CACHE_FP8 && !lat_scale)) return FP8BS_ERR_NULL;
  if (!aligned(latent, 16) || !aligned(rope, 16) ||
      (cache_fmt == FP8BS_CACHE_FP8 && !aligned(lat_scale, 16)))
    return FP8BS_ERR_ALIGN;
  return FP8BS_OK;
}

// [out, out + bytes) meets one of the cache's arrays
static bool over_cache(const void* out, int64_t bytes, const void* latent, const float* lat_scale,
                       const void* rope, int cache_fmt, int64_t P, int64_t ps) {
  const bool fp8 = cache_fmt == FP8BS_CACHE_FP8;
  const int64_t rows = P * ps;
  return overlap(out, bytes, latent, rows * (fp8 ? 512 : 1024)) || overlap(out, bytes, rope, rows * 128) ||
         (fp8 && overlap(out, bytes, lat_scale, rows * 16));
}

// the cache's arrays meet each other (the entry points that write them refuse it)
static bool cache_overlaps(const void* latent, const float* lat_scale, const void* rope, int cache_fmt, int64_t P, int64_t ps) {
  const bool fp8 = cache_fmt == FP8BS_CACHE_FP8;
  const int64_t rows = P * ps, nl = rows * (fp8 ? 512 : 1024);
  return overlap(latent, nl, rope, rows * 128) ||
         (fp8 && (overlap(lat_scale, rows * 16, latent, nl) || overlap(lat_scale, rows * 16, rope, rows * 128)));
}

// elements from the first to the last of a [T, H, width] view with strides ld_t, ld_h, or -1 when beyond int64
static int64_t extent(int64_t T, int64_t H, int64_t ld_t, int64_t ld_h, int64_t width) {
  const int64_t a = mul(T - 1, ld_t), b = mul(H - 1, ld_h);
  if (a < 0 || b < 0 || a > INT64_MAX / 8 || b > INT64_MAX / 8) return -1;
  return a + b + width;
}

int fp8bs_mla_cache_write(const void* q_rope, int64_t ldq_t, int64_t ldq_h, const void* kv,
                          int64_t ld_kv, const void* norm_w, int norm_w_f32, float eps,
                          const float* rope_cs, int64_t n_pos, void* q_out, void* latent,
                          float* lat_scale, void* rope, int cache_fmt, const int32_t* table,
                          const int32_t* cu_q, const int32_t* lens, int64_t T, int64_t H, int64_t B,
                          int64_t W, int64_t P, int64_t ps, int64_t R, int64_t dr, void* stream) {
  if (T < 0 || H < 0 || T > kLimitRows || H > kLimitInt || B > kLimitSeqs || n_pos < 0 || ldq_t < 0 || ldq_h < 0 ||
      ld_kv < 0 || !(eps >= 0.0f && eps <= 3.0e38f))
    return FP8BS_ERR_SHAPE;
  const int64_t nq = mul(mul(T, H), 64);
  if (nq < 0 || mul(nq, 2) < 0 || mul(n_pos, 256) < 0) return FP8BS_ERR_SHAPE;
  if (T == 0 || B == 0) return B < 0 ? FP8BS_ERR_SHAPE : FP8BS_OK;
  if (ldq_t % 8 != 0 || ldq_h % 8 != 0 || ld_kv % 8 != 0) return FP8BS_ERR_ALIGN;
  const int st = cache_checks(latent, lat_scale, rope, cache_fmt, B, W, P, ps, R, dr);
  if (st != FP8BS_OK) return st;
  if (!kv || !norm_w || (n_pos > 0 && !rope_cs) || !table || !cu_q || !lens || (H > 0 && (!q_rope || !q_out)))
    return FP8BS_ERR_NULL;
  if (!aligned(kv, 16) || !aligned(norm_w, norm_w_f32 ? 4 : 2) || !aligned(rope_cs, 4) ||
      !aligned(table, 4) || !aligned(cu_q, 4) || !aligned(lens, 4) ||
      (H > 0 && (!aligned(q_rope, 16) || !aligned(q_out, 16))))
    return FP8BS_ERR_ALIGN;
  const int64_t eq = H > 0 ? extent(T, H, ldq_t, ldq_h, 64) : 0, ek = extent(T, 1, ld_kv, 0, 576);
  if (eq < 0 || ek < 0) return FP8BS_ERR_SHAPE;
  const void* in[] = {q_rope, kv, norm_w, rope_cs, table, cu_q, lens};
  const int64_t size[] = {2 * eq, 2 * ek, norm_w_f32 ? 2048 : 1024, 256 * n_pos, 4 * B * W, 4 * (B + 1), 4 * B};
  for (int i = 0; i < 7; ++i)
    if (overlap(q_out, 2 * nq, in[i], size[i]) ||
        over_cache(in[i], size[i], latent, lat_scale, rope, cache_fmt, P, ps))
      return FP8BS_ERR_ALIAS;
  if (over_cache(q_out, 2 * nq, latent, lat_scale, rope, cache_fmt, P, ps) ||
      cache_overlaps(latent, lat_scale, rope, cache_fmt, P, ps))
    return FP8BS_ERR_ALIAS;
  const fp8bs::MlaCacheWrite a{q_rope, kv, norm_w, rope_cs, q_out, latent, rope, lat_scale, table, cu_q, lens,
                               ldq_t, ldq_h, ld_kv, n_pos, T, H, B, W, P, ps, eps, norm_w_f32 != 0,
                               cache_fmt == FP8BS_CACHE_FP8};
  return status_of(fp8bs::launch_mla_cache_write(a, (hipStream_t)stream));
}

int64_t fp8bs_mla_attention_workspace_size(int64_t T, int64_t H, int64_t B) {
  if (T < 0 || H < 1 || B < 0 || B > 8192) return -1;
  const int64_t rows = mul(T, H);
  if (rows < 0 || rows > kLimitInt) return -1;
  return rows == 0 || B == 0 ? 0 : fp8bs::mla_attention_workspace_bytes(T, H, B);
}

int fp8bs_mla_attention(const void* q_lat, int64_t ldq_t, int64_t ldq_h, const void* q_rope,
                        int64_t ldr_t, int64_t ldr_h, const void* latent, const float* lat_scale,
                        const void* rope, int cache_fmt, const int32_t* table, const int32_t* cu_q,
                        const int32_t* lens, float scale, int causal, void* out, int out_dtype,
                        float* lse, int64_t T, int64_t H, int64_t B, int64_t W, int64_t P,
                        int64_t ps, int64_t R, int64_t dr, void* workspace, int64_t workspace_bytes,
                        void* stream) {
  const int64_t need = fp8bs_mla_attention_workspace_size(T, H, B);
  if (need < 0 || ldq_t < 0 || ldq_h < 0 || ldr_t < 0 || ldr_h < 0 ||
      !(fabsf(scale) <= 2.3e38f))                    // times log2(e) it is still finite
    return FP8BS_ERR_SHAPE;
  if (out_dtype != FP8BS_OUT_BF16 && out_dtype != FP8BS_OUT_F32) return FP8BS_ERR_ENUM;
  if (T == 0 || B == 0) return FP8BS_OK;
  if (workspace_bytes < need) return FP8BS_ERR_SHAPE;
  if (ldq_t % 8 != 0 || ldq_h % 8 != 0 || ldr_t % 8 != 0 || ldr_h % 8 != 0) return FP8BS_ERR_ALIGN;
  const int st = cache_checks(latent, lat_scale, rope, cache_fmt, B, W, P, ps, R, dr);
  if (st != FP8BS_OK) return st;
  if (!q_lat || !q_rope || !table || !cu_q || !lens || !out || (need > 0 && !workspace)) return FP8BS_ERR_NULL;
  if (!aligned(q_lat, 16) || !aligned(q_rope, 16) || !aligned(out, 16) || !aligned(workspace, 16) ||
      !aligned(table, 4) || !aligned(cu_q, 4) || !aligned(lens, 4) || !aligned(lse, 4))
    return FP8BS_ERR_ALIGN;
  const int64_t eq = extent(T, H, ldq_t, ldq_h, 512), er = extent(T, H, ldr_t, ldr_h, 64);
  if (eq < 0 || er < 0) return FP8BS_ERR_SHAPE;
  const int64_t ob = T * H * 512 * (out_dtype == FP8BS_OUT_F32 ? 4 : 2), lb = lse ? 4 * T * H : 0;
  const void* in[] = {q_lat, q_rope, table, cu_q, lens};
  const int64_t size[] = {2 * eq, 2 * er, 4 * B * W, 4 * (B + 1), 4 * B};
  for (int i = 0; i < 5; ++i)
    if (overlap(out, ob, in[i], size[i]) || overlap(lse, lb, in[i], size[i]) ||
        overlap(workspace, need, in[i], size[i]))
      return FP8BS_ERR_ALIAS;
  if (overlap(out, ob, lse, lb) || overlap(workspace, need, out, ob) || overlap(workspace, need, lse, lb) ||
      over_cache(out, ob, latent, lat_scale, rope, cache_fmt, P, ps) ||
      over_cache(lse, lb, latent, lat_scale, rope, cache_fmt, P, ps) ||
      over_cache(workspace, need, latent, lat_scale, rope, cache_fmt, P, ps))
    return FP8BS_ERR_ALIAS;
  const fp8bs::MlaAttention a{q_lat, q_rope, latent, rope, lat_scale, table, cu_q, lens, out, lse, workspace,
                              ldq_t, ldq_h, ldr_t, ldr_h, T, H, B, W, P, ps, scale, causal != 0,
                              out_dtype == FP8BS_OUT_F32, cache_fmt == FP8BS_CACHE_FP8};
  return status_of(fp8bs::launch_mla_attention(a, (hipStream_t)stream));
}

int64_t fp8bs_cache_update_workspace_size(int64_t B, int64_t N, int64_t W, int64_t P) {
  if (P < 1 || P > kLimitInt || N < 0 || N >= (1 << 18) || B < 0 || B > kLimitRows - N || W < 1 || W > kLimitInt)
    return -1;
  return N == 0 ? 0 : fp8bs::cache_update_workspace_bytes(B, N, W, P);
}

int fp8bs_cache_update(void* latent, float* lat_scale, void* rope, int cache_fmt,
                       const int32_t* table, const int32_t* lens, const int32_t* parent,
                       const int32_t* new_lens, int32_t* table_out, int32_t* lens_out, int64_t B,
                       int64_t N, int64_t W, int64_t P, int64_t ps, int64_t R, int64_t dr,
                       void* workspace, int64_t workspace_bytes, void* stream) {
  const int64_t need = fp8bs_cache_update_workspace_size(B, N, W, P);
  if (need < 0) return FP8BS_ERR_SHAPE;
  if (N == 0) return FP8BS_OK;
  if (workspace_bytes < need || mul(N, W) < 0 || mul(mul(N, W), 4) < 0) return FP8BS_ERR_SHAPE;
  const int st = cache_checks(latent, lat_scale, rope, cache_fmt, B, W, P, ps, R, dr);
  if (st != FP8BS_OK) return st;
  if (!parent || !new_lens || !table_out || !lens_out || (need > 0 && !workspace) || (B > 0 && (!table || !lens)))
    return FP8BS_ERR_NULL;
  if (!aligned(workspace, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(parent, 4) ||
      !aligned(new_lens, 4) || !aligned(table_out, 4) || !aligned(lens_out, 4))
    return FP8BS_ERR_ALIGN;
  const void* in[] = {table, lens, parent, new_lens};
  const int64_t is[] = {4 * B * W, 4 * B, 4 * N, 4 * N};
  const void* outs[] = {table_out, lens_out, workspace};
  const int64_t os[] = {4 * N * W, 4 * N, need};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 4; ++i)
      if (overlap(outs[o], os[o], in[i], is[i])) return FP8BS_ERR_ALIAS;
    for (int q = o + 1; q < 3; ++q)
      if (overlap(outs[o], os[o], outs[q], os[q])) return FP8BS_ERR_ALIAS;
    if (over_cache(outs[o], os[o], latent, lat_scale, rope, cache_fmt, P, ps)) return FP8BS_ERR_ALIAS;
  }
  for (int i = 0; i < 4; ++i)
    if (over_cache(in[i], is[i], latent, lat_scale, rope, cache_fmt, P, ps)) return FP8BS_ERR_ALIAS;
  if (cache_overlaps(latent, lat_scale, rope, cache_fmt, P, ps)) return FP8BS_ERR_ALIAS;
  const fp8bs::PageTask a{latent, rope, lat_scale, table, lens, parent, new_lens, table_out, lens_out, nullptr,
                          workspace, B, W, N, P, ps, cache_fmt == FP8BS_CACHE_FP8};
  return status_of(fp8bs::launch_cache_update(a, (hipStream_t)stream));
}

int64_t fp8bs_cache_compact_workspace_size(int64_t B, int64_t W, int64_t P) {
  if (P < 1 || P > kLimitInt || B < 0 || B > kLimitRows || W < 1 || W > kLimitInt) return -1;
  return fp8bs::cache_compact_workspace_bytes(B, W, P);
}

int fp8bs_cache_compact(void* latent, float* lat_scale, void* rope, int cache_fmt,
                        const int32_t* table, const int32_t* lens, int32_t* table_out,
                        int32_t* count, int64_t B, int64_t W, int64_t P, int64_t ps, int64_t R,
                        int64_t dr, void* workspace, int64_t workspace_bytes, void* stream) {
  const int64_t need = fp8bs_cache_compact_workspace_size(B, W, P);
  if (need < 0 || workspace_bytes < need) return FP8BS_ERR_SHAPE;
  const int st = cache_checks(latent, lat_scale, rope, cache_fmt, B, W, P, ps, R, dr);
  if (st != FP8BS_OK) return st;
  if (!count || (need > 0 && !workspace) || (B > 0 && (!table || !lens || !table_out))) return FP8BS_ERR_NULL;
  if (!aligned(workspace, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(table_out, 4) ||
      !aligned(count, 4))
    return FP8BS_ERR_ALIGN;
  const void* in[] = {table, lens};
  const int64_t is[] = {4 * B * W, 4 * B};
  const void* outs[] = {table_out, count, workspace};
  const int64_t os[] = {4 * B * W, 4, need};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 2; ++i)
      if (overlap(outs[o], os[o], in[i], is[i])) return FP8BS_ERR_ALIAS;
    for (int q = o + 1; q < 3; ++q)
      if (overlap(outs[o], os[o], outs[q], os[q])) return FP8BS_ERR_ALIAS;
    if (over_cache(outs[o], os[o], latent, lat_scale, rope, cache_fmt, P, ps)) return FP8BS_ERR_ALIAS;
  }
  for (int i = 0; i < 2; ++i)
    if (over_cache(in[i], is[i], latent, lat_scale, rope, cache_fmt, P, ps)) return FP8BS_ERR_ALIAS;
  if (cache_overlaps(latent, lat_scale, rope, cache_fmt, P, ps)) return FP8BS_ERR_ALIAS;
  const fp8bs::PageTask a{latent, rope, lat_scale, table, lens, nullptr, nullptr, table_out, nullptr, count,
                          workspace, B, W, 0, P, ps, cache_fmt == FP8BS_CACHE_FP8};
  return status_of(fp8bs::launch_cache_compact(a, (hipStream_t)stream));
}

}  // extern "C"
