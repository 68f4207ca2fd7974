// swiglu.hip -- the activation between the two products of an expert,
//   a = g * sigmoid(g) * u,
// with block-scaled FP8 output for the second product (act_quant's rule:
// "DeepSeek-V3 Administrator & Developer Guide" 8.5.1) or bf16, and its gradient.
// HBM-bound: every element is read and written once; 16 consecutive lanes hold a
// block of 128.
#include "device_common.h"
#include "launch.h"

namespace fp8bs {

namespace {

constexpr int kThreads = 256;
constexpr int kPasses = 4;           // vectors of 8 elements that a thread takes

// Where thread i of a run of vectors lies: rows of nv vectors, the run starting at row
// `row`, vector `col`.  Less than 2^31 vectors behind it.
struct Run {
  int64_t row;
  uint32_t col, nv;
};
__device__ __forceinline__ Run run_of(int64_t first, int64_t nv) {
  const int64_t r = first / nv;      // the same for the workgroup
  return {r, (uint32_t)(first - r * nv), (uint32_t)nv};
}
__device__ __forceinline__ void place(const Run& run, uint32_t i, int64_t* row, uint32_t* col) {
  const uint32_t at = run.col + i;   // nv < 2^28 and i < 2^10
  const uint32_t down = at / run.nv;
  *row = run.row + down;
  *col = at - down * run.nv;
}

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]), pack2_bf16(f[4], f[5]), pack2_bf16(f[6], f[7]));
}

__device__ __forceinline__ float sigmoid(float x) { return __fdiv_rn(1.0f, 1.0f + expf(-x)); }

// rows that the call has: all, or fewer by the device's count
__device__ __forceinline__ int64_t rows_of(const int32_t* n_rows, int64_t M) {
  return n_rows ? min(max<int64_t>(*n_rows, 0), M) : M;
}

}  // namespace

__global__ __launch_bounds__(kThreads) void swiglu_kernel(const SwiGlu p) {
  const int64_t nv = p.N / 8, rows = rows_of(p.n_rows, p.M);
  const Run run = run_of((int64_t)blockIdx.x * (kThreads * kPasses), nv);
  if (run.row >= rows) return;
  uint4 g[kPasses], u[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    int64_t r;
    uint32_t c;
    place(run, threadIdx.x + k * kThreads, &r, &c);
    r = min(r, rows - 1);
    g[k] = *((const uint4*)((const uint16_t*)p.gate + r * p.ld_g) + c);
    u[k] = *((const uint4*)((const uint16_t*)p.up + r * p.ld_u) + c);
  }
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    int64_t r;
    uint32_t c;
    place(run, threadIdx.x + k * kThreads, &r, &c);
    if (r >= rows) return;                                   // blocks of 128 lie in one row: 16 lanes go together
    float a[8], b[8];
    unpack8(g[k], a);
    unpack8(u[k], b);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = a[i] * sigmoid(a[i]) * b[i];
    const int64_t at = r * nv + c;
    if (p.y) store_nt((uint4*)p.y + at, pack8(a));
    if (p.q) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, f32_bits(a[i]) & 0x7FFFFFFFu);
      top = row16_max_u32(top);
      const float sc = p.ue8m0 ? block_scale<true>(bits_f32(top)) : block_scale<false>(bits_f32(top));
      const float rs = __fdiv_rn(1.0f, sc);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = div_markstein(a[i], sc, rs);
      store_nt((uint2*)p.q + at, make_uint2(pack4_e4m3(a[0], a[1], a[2], a[3]), pack4_e4m3(a[4], a[5], a[6], a[7])));
      if ((threadIdx.x & 15) == 0) p.s[at / 16] = sc;
    }
  }
}

// du = dy * g * sigmoid(g),  dg = dy * u * sigmoid(g) * (1 + g * (1 - sigmoid(g)))
__global__ __launch_bounds__(kThreads) void swiglu_bwd_kernel(const SwiGluBwd p) {
  const int64_t nv = p.N / 8, rows = rows_of(p.n_rows, p.M);
  const Run run = run_of((int64_t)blockIdx.x * (kThreads * kPasses), nv);
  if (run.row >= rows) return;
  uint4 g[kPasses], u[kPasses], d[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    int64_t r;
    uint32_t c;
    place(run, threadIdx.x + k * kThreads, &r, &c);
    r = min(r, rows - 1);
    g[k] = *((const uint4*)((const uint16_t*)p.gate + r * p.ld_g) + c);
    u[k] = *((const uint4*)((const uint16_t*)p.up + r * p.ld_u) + c);
    d[k] = ((const uint4*)p.dy)[r * nv + c];
  }
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    int64_t r;
    uint32_t c;
    place(run, threadIdx.x + k * kThreads, &r, &c);
    if (r >= rows) return;
    float a[8], b[8], e[8];
    unpack8(g[k], a);
    unpack8(u[k], b);
    unpack8(d[k], e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(a[i]), x = e[i] * s;
      e[i] = x * b[i] * __builtin_fmaf(a[i], 1.0f - s, 1.0f);
      b[i] = x * a[i];
    }
    store_nt((uint4*)((uint16_t*)p.dgate + r * p.ld_dg) + c, pack8(e));
    store_nt((uint4*)((uint16_t*)p.dup + r * p.ld_du) + c, pack8(b));
  }
}

// One launch: at most 2^32 - 1 threads, kPasses vectors of 8 a thread.
bool swiglu_fits(int64_t M, int64_t N) {
  if (M <= 0 || N <= 0) return true;
  const int64_t most = (((int64_t)1 << 32) - 1) / kThreads * (kThreads * kPasses);
  return N < ((int64_t)1 << 31) && M <= most / (N / 8);
}

static dim3 grid_of(int64_t M, int64_t N) {
  return dim3((unsigned)((M * (N / 8) + kThreads * kPasses - 1) / (kThreads * kPasses)));
}

hipError_t launch_swiglu(const SwiGlu& p, hipStream_t stream) {
  swiglu_kernel<<<grid_of(p.M, p.N), dim3(kThreads), 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const SwiGluBwd& p, hipStream_t stream) {
  swiglu_bwd_kernel<<<grid_of(p.M, p.N), dim3(kThreads), 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace fp8bs
