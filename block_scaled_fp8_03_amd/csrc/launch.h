// launch.h -- internal kernel launchers (host side).  Arguments have been
// validated by the C ABI layer before these are called; each returns the
// hipError_t of its launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bs {

// Whether one act_quant (or moe_quant_scatter) launch covers `rows` rows of
// K columns (its grid's thread limit).
bool act_quant_fits(int64_t rows, int64_t K);
hipError_t launch_act_quant(const void* x, void* q, float* s, int64_t M, int64_t K, bool ue8m0,
                            hipStream_t stream);
// The float32 -> e4m3 conversion of act_quant / weight_quant on its own.
bool e4m3_encode_fits(int64_t n);
hipError_t launch_e4m3_encode(const float* x, void* q, int64_t n, hipStream_t stream);
hipError_t launch_weight_quant(const void* w, void* q, float* s, int64_t N, int64_t K, bool ue8m0,
                               hipStream_t stream);
// Whether one weight_dequant launch covers [N, K] (its grid's thread limit).
bool weight_dequant_fits(int64_t N, int64_t K);
hipError_t launch_weight_dequant(const void* w, const float* s, void* y, int64_t N, int64_t K,
                                 hipStream_t stream);
hipError_t launch_gemm(const void* a, const float* a_s, const void* b, const float* b_s, void* c,
                       int64_t M, int64_t N, int64_t K, bool out_f32, hipStream_t stream);
hipError_t launch_moe_gemm(const void* a, const float* a_s, const void* b, const float* b_s,
                           const int32_t* offsets, void* c, int64_t R, int64_t E, int64_t N,
                           int64_t K, bool out_f32, hipStream_t stream);

hipError_t launch_gemm_ue8m0(const void* a, const float* a_s, const void* b, const float* b_s,
                             void* c, int64_t M, int64_t N, int64_t K, bool out_f32,
                             hipStream_t stream);
hipError_t launch_w8a16_gemm(const void* x, const void* w, const float* w_s, void* c, int64_t M,
                             int64_t N, int64_t K, bool out_f32, hipStream_t stream);
hipError_t launch_moe_quant_scatter(const void* x, const int32_t* row_of, void* q, float* s,
                                    int64_t T, int64_t topk, int64_t R, int64_t K, bool ue8m0,
                                    hipStream_t stream);
int64_t moe_route_workspace_bytes(int64_t T, int64_t topk, int64_t E);
hipError_t launch_moe_route(const int32_t* indices, int64_t T, int64_t topk, int64_t E,
                            int32_t* offsets, int32_t* row_token, int32_t* row_of, void* workspace,
                            hipStream_t stream);
// fp8bs_moe_route_noalloc: the count table in a file-scope device array of
// kRouteScratchBytes per GPU instead of a caller workspace.
constexpr int64_t kRouteScratchBytes = (int64_t)1 << 20;
hipError_t launch_moe_route_noalloc(const int32_t* indices, int64_t T, int64_t topk, int64_t E,
                                    int32_t* offsets, int32_t* row_token, int32_t* row_of,
                                    hipStream_t stream);
hipError_t launch_moe_combine(const void* out, const float* w, const int32_t* row_of, void* y,
                              int64_t T, int64_t topk, int64_t R, int64_t N, bool out_f32,
                              hipStream_t stream);
hipError_t launch_moe_combine_bwd(const void* dy, const void* out, const float* w, const int32_t* row_of, void* d_out,
                                  float* d_w, int64_t T, int64_t topk, int64_t R, int64_t N, bool dy_f32,
                                  hipStream_t stream);
hipError_t launch_mla_absorb_key(const void* q, int64_t ld_t, int64_t ld_h, const void* w,
                                 const float* ws, void* out, int64_t T, int64_t H, int64_t dn,
                                 int64_t dv, int64_t R, bool out_f32, hipStream_t stream);
hipError_t launch_mla_absorb_value(const void* x, int64_t ld_t, int64_t ld_h, const void* w,
                                   const float* ws, void* out, int64_t T, int64_t H, int64_t dn,
                                   int64_t dv, int64_t R, bool out_f32, hipStream_t stream);

// fp8bs_mla_attention's arguments
struct MlaAttention {
  const void *q_lat, *q_rope, *latent, *rope;
  const float* lat_scale;
  const int32_t *table, *cu_q, *lens;
  void* out;
  float* lse;
  void* workspace;
  int64_t ldq_t, ldq_h, ldr_t, ldr_h;
  int64_t T, H, B, W, P, ps;
  float scale;
  bool causal, out_f32, fp8;
};
hipError_t launch_mla_attention(const MlaAttention& a, hipStream_t stream);
int64_t mla_attention_workspace_bytes(int64_t T, int64_t H, int64_t B);

// fp8bs_mla_cache_write's arguments
struct MlaCacheWrite {
  const void *q, *kv, *w;
  const float* cs;
  void *q_out, *latent, *rope;
  float* scale;
  const int32_t *table, *cu_q, *lens;
  int64_t ldq_t, ldq_h, ld_kv, n_pos;
  int64_t T, H, B, W, P, ps;
  float eps;
  bool w_f32, fp8;
};
hipError_t launch_mla_cache_write(const MlaCacheWrite& a, hipStream_t stream);

// fp8bs_cache_update's and fp8bs_cache_compact's arguments (update: parent, new_lens, lens_out; compact: count)
struct PageTask {
  void *latent, *rope, *scale;
  const int32_t *table, *lens, *parent, *new_lens;
  int32_t *table_out, *lens_out, *count;
  void* workspace;
  int64_t B, W, N, P, ps;
  bool fp8;
};
int64_t cache_update_workspace_bytes(int64_t B, int64_t N, int64_t W, int64_t P);
int64_t cache_compact_workspace_bytes(int64_t B, int64_t W, int64_t P);
hipError_t launch_cache_update(const PageTask& a, hipStream_t stream);
hipError_t launch_cache_compact(const PageTask& a, hipStream_t stream);

// Calls that move at least this many bytes read their inputs with the non-temporal hint;
// below, what the call before left in the Infinity Cache (256 MB) is found there, which
// the hint gives up.  us, with the hint / without (inputs of three calls in turn):
// SwiGLU 84 MB 16.9 / 16.1, 169 MB 29.8 / 32.4, 338 MB 56.1 / 61.3; its gradient 84 MB
// 14.5 / 13.4, 168 MB 27.2 / 28.6; RMSNorm 132 MB 25.4 / 21.3, 265 MB 46.2 / 47.0; the
// combine's gradient 98 MB 24.6 / 18.1, 196 MB 48.5 / 51.4, 999 MB 190 / 203.  Rows that a
// count on the device leaves out count too: 2000 of 32768 rows of 2048, SwiGLU 5.7 / 6.6, its
// gradient 8.1 / 8.2.
constexpr int64_t kHintBytes = (int64_t)160 << 20;

// fp8bs_rmsnorm's arguments (res and res_out, y, q and s: NULL where there is none)
struct RmsNorm {
  const void *x, *res, *w;
  void *res_out, *y, *q;
  float* s;
  int64_t ld_x, M, K;
  float eps;
  bool res_f32, w_f32, ue8m0;
};
bool rmsnorm_fits(int64_t M, int64_t K);
hipError_t launch_rmsnorm(const RmsNorm& p, hipStream_t stream);

// fp8bs_rmsnorm_bwd's arguments (h and dx, dres: of h's type)
struct RmsNormBwd {
  const void *dy, *h, *w, *dres;
  void* dx;
  float* dw;
  void* workspace;
  int64_t ld_h, M, K;
  float eps;
  bool h_f32, w_f32;
};
int64_t rmsnorm_bwd_workspace_bytes(int64_t M, int64_t K);
hipError_t launch_rmsnorm_bwd(const RmsNormBwd& p, hipStream_t stream);

// fp8bs_moe_gate's, fp8bs_moe_balance's and fp8bs_moe_gate_bwd's arguments
struct MoeGate {
  const void* logits;
  const float* bias;
  int32_t* indices;
  float* weights;
  int64_t ld, T, E, topk, groups, keep;
  float route_scale;
  bool f32, softmax, normalize;
  bool bias_wide;          // the bias is aligned to 16 bytes
};
hipError_t launch_moe_gate(const MoeGate& p, hipStream_t stream);
struct MoeBalance {
  const void* logits;
  const int32_t *indices, *cu;
  int32_t* counts;
  float *probs, *loss;
  void* workspace;
  int64_t ld, T, S, E, topk;
  bool f32, softmax;
  float* part_probs;       // in the workspace
  int32_t* part_counts;
};
int64_t moe_balance_workspace_bytes(int64_t T, int64_t S, int64_t E);
hipError_t launch_moe_balance(const MoeBalance& p, hipStream_t stream);
struct MoeGateBwd {
  const void* logits;
  const int32_t *indices, *cu, *counts;
  const float *d_weights, *d_loss;
  void* d_logits;
  int64_t ld, T, S, E, topk;
  float route_scale;
  bool f32, softmax, normalize, out_f32;
};
hipError_t launch_moe_gate_bwd(const MoeGateBwd& p, hipStream_t stream);

// fp8bs_swiglu's and fp8bs_swiglu_bwd's arguments
struct SwiGlu {
  const void *gate, *up;
  const int32_t* n_rows;
  void *y, *q;
  float* s;
  int64_t ld_g, ld_u, M, N;
  bool ue8m0;
};
struct SwiGluBwd {
  const void *dy, *gate, *up;
  const int32_t* n_rows;
  void *dgate, *dup;
  int64_t ld_g, ld_u, ld_dg, ld_du, M, N;
};
bool swiglu_fits(int64_t M, int64_t N);
hipError_t launch_swiglu(const SwiGlu& p, hipStream_t stream);
hipError_t launch_swiglu_bwd(const SwiGluBwd& p, hipStream_t stream);

}  // namespace fp8bs
