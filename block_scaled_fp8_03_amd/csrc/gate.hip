// gate.hip -- the gate of a block with experts ("DeepSeek-V3 Administrator &
// Developer Guide" 8.4: scores, groups, top-k, normalised and scaled weights), the
// balance loss over its scores, and the gradient of both by the logits.
//
// One wave a token: lane l holds experts l*V .. l*V + V - 1, so the lowest lane
// and the lowest register of a maximum are the lowest expert.
#include <algorithm>

#include "device_common.h"
#include "launch.h"

namespace fp8bs {

namespace {

constexpr int kWaves = 4;            // tokens that a workgroup of the gate takes

__device__ __forceinline__ float minus_inf() { return bits_f32(0xFF800000u); }

// Sum over a wave, the same order everywhere; every lane receives it.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) v += __shfl_xor(v, i);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) v += __shfl_xor(v, i);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) v = fmaxf(v, __shfl_xor(v, i));
  return v;
}

// Floats as unsigned numbers of the same order, above 0; -0 and 0 alike.
__device__ __forceinline__ uint32_t order_of(float f) {
  const uint32_t b = f32_bits(f + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t k) {
  return bits_f32(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}

// The token's logits: z[v] of expert lane*V + v; one that is masked (-inf), NaN or
// behind the last expert gives -inf.
template <int V>
__device__ __forceinline__ void load_logits(const void* logits, bool f32, int64_t at, int E, int lane, float* z) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane * V + v;
    float f = minus_inf();
    if (e < E) f = f32 ? ((const float*)logits)[at + e] : bits_f32((uint32_t)((const uint16_t*)logits)[at + e] << 16);
    z[v] = f > minus_inf() ? f : minus_inf();
  }
}

// score[v] in 64 bits, rounded once; 0 for masked experts (all of a token masked: all 0).
// Two scores that float32 arithmetic would leave a rounding apart, or exchange, decide
// which expert a token takes, so they are computed where that cannot happen.
template <int V>
__device__ __forceinline__ void exact_scores(const float* z, bool softmax, float* score) {
  if (!softmax) {
#pragma unroll
    for (int v = 0; v < V; ++v) score[v] = (float)(1.0 / (1.0 + exp(-(double)z[v])));
    return;
  }
  float top = z[0];
#pragma unroll
  for (int v = 1; v < V; ++v) top = fmaxf(top, z[v]);
  top = wave_max(top);
  double e[V], sum = 0.0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    e[v] = z[v] == minus_inf() ? 0.0 : z[v] == top ? 1.0 : exp((double)z[v] - (double)top);
    sum += e[v];
  }
  sum = wave_sum(sum);
#pragma unroll
  for (int v = 0; v < V; ++v) score[v] = sum > 0.0 ? (float)(e[v] / sum) : 0.0f;
}

// score[v] in float32, and the sum of all of them (1 for a softmax, 0 where all are masked).
template <int V>
__device__ __forceinline__ float scores(const float* z, bool softmax, float* score) {
  float sum = 0.0f;
  if (!softmax) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      // the exponential of what is below 0 alone: scores go down to float32's smallest numbers
      const float x = expf(-fabsf(z[v]));
      score[v] = __fdiv_rn(z[v] < 0.0f ? x : 1.0f, 1.0f + x);
      sum += score[v];
    }
    return wave_sum(sum);
  }
  float top = z[0];
#pragma unroll
  for (int v = 1; v < V; ++v) top = fmaxf(top, z[v]);
  top = wave_max(top);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    score[v] = z[v] == minus_inf() ? 0.0f : z[v] == top ? 1.0f : expf(z[v] - top);
    sum += score[v];
  }
  sum = wave_sum(sum);
  const float by = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) score[v] *= by;
  return sum > 0.0f ? 1.0f : 0.0f;
}

// score[v] over their sum; a softmax's are that already.  A quotient, not a product
// with 1 / sum: that is infinite for the sum of the smallest scores.
template <int V>
__device__ __forceinline__ void shares(float* score, float sum, bool softmax) {
  if (softmax) return;
#pragma unroll
  for (int v = 0; v < V; ++v) score[v] = sum > 0.0f ? __fdiv_rn(score[v], sum) : 0.0f;
}

}  // namespace

// ----------------------------------------------------------------------------
// gate
// ----------------------------------------------------------------------------
template <int V>
__global__ __launch_bounds__(64 * kWaves) void moe_gate_kernel(const MoeGate p) {
  __shared__ uint32_t keys[kWaves][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t >= p.T) return;                                       // waves work apart: no barrier follows
  const int E = (int)p.E, G = (int)p.groups, size = E / G;
  float z[V], score[V];
  load_logits<V>(p.logits, p.f32, t * p.ld, E, lane, z);
  uint32_t key[V];
  if (p.bias) {
    exact_scores<V>(z, p.softmax, score);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane * V + v;
      const float k = score[v] + (e < E ? p.bias[e] : 0.0f);
      key[v] = z[v] > minus_inf() && k > minus_inf() ? order_of(k) : 0;
    }
  } else {
    scores<V>(z, p.softmax, score);
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = z[v] > minus_inf() ? order_of(z[v]) : 0;
  }
  if (G > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) keys[wave][lane * V + v] = key[v];
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
    // lane g: the value of group g
    uint32_t value = 0;
    if (lane < G) {
      uint32_t a = 0, b = 0;
      for (int i = 0; i < size; ++i) {
        const uint32_t k = keys[wave][lane * size + i];
        b = max(b, min(a, k));
        a = max(a, k);
      }
      value = p.bias && b ? order_of(float_of(a) + float_of(b)) : a;
    }
    int before = 0;                                           // groups that come before this one
    for (int g = 0; g < G; ++g) {
      const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)value, g);
      before += o > value || (o == value && g < lane);
    }
    const uint64_t kept = __ballot(lane < G && before < (int)p.keep);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int g = min((lane * V + v) / size, G - 1);
      if (!(kept >> g & 1)) key[v] = 0;
    }
  }
  int id = -1;
  float w = 0.0f;
  for (int k = 0; k < (int)p.topk; ++k) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int v = 1; v < V; ++v)
      if (key[v] > best) best = key[v], at = v;
    const uint32_t top = wave_max_u32(best);
    if (top == 0) break;                                      // no expert is left
    const int who = __ffsll((unsigned long long)__ballot(best == top)) - 1;
    float s = score[0];
#pragma unroll
    for (int v = 1; v < V; ++v)
      if (v == at) s = score[v];
    const int e = who * V + __builtin_amdgcn_readlane(at, who);
    s = bits_f32((uint32_t)__builtin_amdgcn_readlane((int)f32_bits(s), who));
    if (lane == k) id = e, w = s;
    if (lane == who) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v == at) key[v] = 0;
    }
  }
  if (p.normalize) {
    const float sum = wave_sum(w);
    w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
  }
  if (lane < (int)p.topk) {
    p.indices[t * p.topk + lane] = id;
    p.weights[t * p.topk + lane] = w * p.route_scale;
  }
}

// V registers a lane for E experts
#define FP8BS_BY_EXPERTS(E, CALL)      \
  if ((E) <= 64) { CALL(1); }          \
  else if ((E) <= 128) { CALL(2); }    \
  else if ((E) <= 256) { CALL(4); }    \
  else if ((E) <= 512) { CALL(8); }    \
  else { CALL(16); }

hipError_t launch_moe_gate(const MoeGate& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + kWaves - 1) / kWaves)), block(64 * kWaves);
#define CALL(V) moe_gate_kernel<V><<<grid, block, 0, stream>>>(p)
  FP8BS_BY_EXPERTS(p.E, CALL)
#undef CALL
  return hipGetLastError();
}

// ----------------------------------------------------------------------------
// balance: workgroup (c, s) takes part c of sequence s's tokens, one a wave at a
// time; a lane adds its experts' shares up in registers.  The second kernel adds
// the parts in order and makes the loss; one part needs none.
// ----------------------------------------------------------------------------
namespace {

constexpr int kBalanceWaves = 8;
constexpr int kBalanceRows = 64;     // tokens that a part is meant to have
constexpr int kBalanceParts = 2048;  // workgroups that more parts are not worth

int64_t balance_parts(int64_t T, int64_t S) {
  const int64_t by_rows = (T + kBalanceRows - 1) / kBalanceRows;
  return std::max<int64_t>(1, std::min<int64_t>(by_rows, kBalanceParts / std::max<int64_t>(S, 1)));
}

// Sequence s's tokens [a, b), inside [0, T)
__device__ __forceinline__ void bounds_of(const int32_t* cu, int64_t s, int64_t T, int64_t* a, int64_t* b) {
  *a = cu ? min(max<int64_t>(cu[s], 0), T) : 0;
  *b = cu ? max(min(max<int64_t>(cu[s + 1], 0), T), *a) : T;
}

// loss of one sequence, by the first wave: E / (topk * n) * sum counts * probs
__device__ __forceinline__ void write_loss(float part, int64_t n, const MoeBalance& p, int64_t s) {
  part = wave_sum(part);
  if (threadIdx.x == 0) p.loss[s] = n > 0 ? part * __fdiv_rn((float)p.E, (float)p.topk * (float)n) : 0.0f;
}

}  // namespace

template <int V>
__global__ __launch_bounds__(64 * kBalanceWaves) void moe_balance_kernel(const MoeBalance p, int64_t parts) {
  __shared__ float sums[kBalanceWaves][64 * V];
  __shared__ int32_t hits[64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t s = blockIdx.x / parts, c = blockIdx.x % parts;
  const int E = (int)p.E;
  for (int i = threadIdx.x; i < 64 * V; i += 64 * kBalanceWaves) hits[i] = 0;
  __syncthreads();
  int64_t a, b;
  bounds_of(p.cu, s, p.T, &a, &b);
  const int64_t n = b - a, lo = a + n * c / parts, hi = a + n * (c + 1) / parts;
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  for (int64_t t = lo + wave; t < hi; t += kBalanceWaves) {
    float z[V], score[V];
    load_logits<V>(p.logits, p.f32, t * p.ld, E, lane, z);
    const float sum = scores<V>(z, p.softmax, score);
    shares<V>(score, sum, p.softmax);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] += score[v];
    for (int k = lane; k < (int)p.topk; k += 64) {
      const int32_t e = p.indices[t * p.topk + k];
      if (e >= 0 && e < E) atomicAdd(&hits[e], 1);            // whole numbers: any order gives the same
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) sums[wave][lane * V + v] = acc[v];
  __syncthreads();
  const float mean = n > 0 ? __fdiv_rn(1.0f, (float)n) : 0.0f;
  float* pr = parts > 1 ? p.part_probs + (s * parts + c) * p.E : p.probs + s * p.E;
  int32_t* co = parts > 1 ? p.part_counts + (s * parts + c) * p.E : p.counts + s * p.E;
  for (int e = threadIdx.x; e < E; e += 64 * kBalanceWaves) {
    float q = 0.0f;
    for (int w = 0; w < kBalanceWaves; ++w) q += sums[w][e];
    if (parts == 1) q *= mean;
    pr[e] = q;
    co[e] = hits[e];
    sums[0][e] = q * (float)hits[e];
  }
  if (parts > 1) return;
  __syncthreads();
  if (wave == 0) {
    float part = 0.0f;
    for (int e = lane; e < E; e += 64) part += sums[0][e];
    write_loss(part, n, p, s);
  }
}

__global__ __launch_bounds__(256) void moe_balance_join_kernel(const MoeBalance p, int64_t parts) {
  __shared__ float red[1024];
  const int64_t s = blockIdx.x;
  const int E = (int)p.E;
  int64_t a, b;
  bounds_of(p.cu, s, p.T, &a, &b);
  const int64_t n = b - a;
  const float mean = n > 0 ? __fdiv_rn(1.0f, (float)n) : 0.0f;
  for (int e = threadIdx.x; e < E; e += 256) {
    float q = 0.0f;
    int32_t h = 0;
    for (int64_t c = 0; c < parts; ++c) {
      q += p.part_probs[(s * parts + c) * p.E + e];
      h += p.part_counts[(s * parts + c) * p.E + e];
    }
    q *= mean;
    p.probs[s * p.E + e] = q;
    p.counts[s * p.E + e] = h;
    red[e] = q * (float)h;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    float part = 0.0f;
    for (int e = threadIdx.x; e < E; e += 64) part += red[e];
    write_loss(part, n, p, s);
  }
}

int64_t moe_balance_workspace_bytes(int64_t T, int64_t S, int64_t E) {
  const int64_t parts = balance_parts(T, S);
  return parts > 1 ? 8 * S * parts * E : 0;
}

hipError_t launch_moe_balance(const MoeBalance& q, hipStream_t stream) {
  MoeBalance p = q;
  const int64_t parts = balance_parts(p.T, p.S);
  p.part_probs = (float*)p.workspace;
  p.part_counts = (int32_t*)p.workspace + p.S * parts * p.E;
  const dim3 grid((unsigned)(p.S * parts)), block(64 * kBalanceWaves);
#define CALL(V) moe_balance_kernel<V><<<grid, block, 0, stream>>>(p, parts)
  FP8BS_BY_EXPERTS(p.E, CALL)
#undef CALL
  if (parts > 1) moe_balance_join_kernel<<<dim3((unsigned)p.S), dim3(256), 0, stream>>>(p, parts);
  return hipGetLastError();
}

// ----------------------------------------------------------------------------
// gradient by the logits, by way of u_i = score_i * dL / d score_i, in which no
// quotient of small scores is infinite:
//   the loss of the token's sequence (counts constant), over share_i = score_i / sum:
//     g_i = d_loss * E / (topk * n^2) * counts_i,  u_i = (g_i - sum_j g_j share_j) share_i
//   the weights w_k = scale * score_k / S (S the chosen scores' sum):
//     u_k += scale * (dw_k - sum_j dw_j score_j / S) score_k / S
//     (not normalised: scale * dw_k score_k)
//   sigmoid: dz_i = u_i (1 - score_i);  softmax: dz_i = u_i - score_i sum_j u_j
// ----------------------------------------------------------------------------
template <int V>
__global__ __launch_bounds__(64 * kWaves) void moe_gate_bwd_kernel(const MoeGateBwd p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t >= p.T) return;
  const int E = (int)p.E;
  float z[V], score[V], u[V];
  load_logits<V>(p.logits, p.f32, t * p.ld, E, lane, z);
  const float sum = scores<V>(z, p.softmax, score);
#pragma unroll
  for (int v = 0; v < V; ++v) u[v] = 0.0f;
  if (p.d_loss) {
    // the sequence that holds t: the last with cu[s] <= t
    int64_t s = 0;
    if (p.cu) {
      int64_t hi = p.S;
      while (hi - s > 1) {
        const int64_t mid = (s + hi) / 2;
        if (p.cu[mid] <= t) s = mid;
        else hi = mid;
      }
    }
    int64_t a, b;
    bounds_of(p.cu, s, p.T, &a, &b);
    if (t >= a && t < b && sum > 0.0f) {
      const float n = (float)(b - a);
      const float c = __fdiv_rn(__fdiv_rn(p.d_loss[s] * (float)E, (float)p.topk * n), n);
      float share[V], mean = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) share[v] = score[v];
      shares<V>(share, sum, p.softmax);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        u[v] = e < E ? c * (float)p.counts[s * p.E + e] : 0.0f;
        mean = __builtin_fmaf(u[v], share[v], mean);
      }
      mean = wave_sum(mean);
#pragma unroll
      for (int v = 0; v < V; ++v) u[v] = (u[v] - mean) * share[v];
    }
  }
  if (p.d_weights) {
    const int K = (int)p.topk;
    int e = -1;
    float uk = 0.0f, own = 0.0f;
    if (lane < K) {
      e = p.indices[t * p.topk + lane];
      uk = p.d_weights[t * p.topk + lane];
      if (e < 0 || e >= E) e = -1;
    }
    // lane k: the score of the token's k-th expert
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float o = __shfl(score[v], e < 0 ? 0 : e / V);
      if (e >= 0 && e % V == v) own = o;
    }
    if (e < 0) uk = 0.0f;
    if (p.normalize) {
      const float S = wave_sum(own);
      own = S > 0.0f ? __fdiv_rn(own, S) : 0.0f;
      uk -= wave_sum(uk * own);
    }
    uk *= p.route_scale * own;
    for (int k = 0; k < K; ++k) {                             // one after the other: an id may be there twice
      const int ek = __builtin_amdgcn_readlane(e, k);
      const float add = bits_f32((uint32_t)__builtin_amdgcn_readlane((int)f32_bits(uk), k));
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (ek == lane * V + v) u[v] += add;
    }
  }
  float all = 0.0f;
  if (p.softmax) {
#pragma unroll
    for (int v = 0; v < V; ++v) all += u[v];
    all = wave_sum(all);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane * V + v;
    if (e >= E) continue;
    float dz;
    if (p.softmax) {
      dz = __builtin_fmaf(-score[v], all, u[v]);
    } else {
      const float x = expf(-fabsf(z[v]));                     // 1 - score without the cancellation near 1
      dz = u[v] * __fdiv_rn(z[v] < 0.0f ? 1.0f : x, 1.0f + x);
    }
    if (p.out_f32) ((float*)p.d_logits)[t * p.E + e] = dz;
    else ((uint16_t*)p.d_logits)[t * p.E + e] = (uint16_t)pack2_bf16(dz, 0.0f);
  }
}

hipError_t launch_moe_gate_bwd(const MoeGateBwd& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + kWaves - 1) / kWaves)), block(64 * kWaves);
#define CALL(V) moe_gate_bwd_kernel<V><<<grid, block, 0, stream>>>(p)
  FP8BS_BY_EXPERTS(p.E, CALL)
#undef CALL
  return hipGetLastError();
}

}  // namespace fp8bs
