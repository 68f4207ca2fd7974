// gate.hip -- the gate of a block with experts ("DeepSeek-V3 Administrator &
// Developer Guide" 8.4: scores, groups, top-k, normalised and scaled weights), the
// balance loss over its scores, and the gradient of both by the logits.
//
// One wave a token: lane l holds experts l*V .. l*V + V - 1, so the lowest lane
// and the lowest register of a maximum are the lowest expert.  A token's logits are
// a few hundred bytes: what these kernels take is a wave's chain of instructions
// (few tokens) or the instructions of all waves (many), not HBM.  256 experts in 8
// groups, top 8, from a graph: 32 tokens 4.1 us, 1.6 of it the launch, 4096 tokens 6.3,
// 30000 tokens 29 (564 vector instructions a token, 8 x 33 of them the choice, 108 the
// scores); counts, loss and both gradients of 4096 tokens 15.8.
#include <algorithm>

#include "device_common.h"
#include "launch.h"

namespace fp8bs {

namespace {

constexpr int kWaves = 4;            // tokens that a workgroup of the gate takes

__device__ __forceinline__ float minus_inf() { return bits_f32(0xFF800000u); }

__device__ __forceinline__ float wave_max(float v) {
  uint32_t b = f32_bits(v);
  b ^= (uint32_t)((int32_t)b >> 31) | 0x80000000u;           // of the same order as unsigned numbers
  b = wave_max_uniform(b);
  return bits_f32(b ^ ((uint32_t)((int32_t)~b >> 31) | 0x80000000u));
}
// Not by the name of the sum of floats, which it would hide from what stands in this namespace
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) v += __shfl_xor(v, i);
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

// V consecutive 4-byte words from e on, as wide as they go; `fill` behind E.  VEC: V
// divides E and the address is aligned to V words.
template <int V, bool VEC>
__device__ __forceinline__ void load_words(const uint32_t* p, int e, int E, uint32_t fill, uint32_t* w) {
  if (VEC && V == 2) {
    const uint2 u = e < E ? *(const uint2*)(p + e) : make_uint2(fill, fill);
    w[0] = u.x, w[V > 1 ? 1 : 0] = u.y;
  } else if (VEC && V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const uint4 u = e < E ? *(const uint4*)(p + e + i) : make_uint4(fill, fill, fill, fill);
      w[i] = u.x, w[(i + 1) % V] = u.y, w[(i + 2) % V] = u.z, w[(i + 3) % V] = u.w;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] = e + v < E ? p[e + v] : fill;
  }
}

// The token's logits: z[v] of expert lane*V + v; one that is masked (-inf), NaN or
// behind the last expert gives -inf.
template <int V, bool VEC>
__device__ __forceinline__ void load_logits(const void* logits, bool f32, int64_t at, int E, int lane, float* z) {
  const int e = lane * V;
  if (f32) {
    uint32_t w[V];
    load_words<V, VEC>((const uint32_t*)logits + at, e, E, 0xFF800000u, w);
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] = bits_f32(w[v]);
  } else if (VEC && V > 1) {
    constexpr int W = V / 2 > 0 ? V / 2 : 1;                  // two logits a word
    uint32_t w[W];
    load_words<W, true>((const uint32_t*)((const uint16_t*)logits + at), lane * W, E / 2, 0xFF80FF80u, w);
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] = v % 2 ? bf16_hi(w[v / 2]) : bf16_lo(w[v / 2]);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      z[v] = e + v < E ? bits_f32((uint32_t)((const uint16_t*)logits)[at + e + v] << 16) : minus_inf();
  }
#pragma unroll
  for (int v = 0; v < V; ++v) z[v] = z[v] > minus_inf() ? z[v] : minus_inf();
}

// e^x for -150 <= x <= 0 in 64 bits, within 2^-36 of it: x = n ln 2 + r, |r| <= ln 2 / 2,
// the exponential series of r to r^9 (what is left out is below 2^-37).  n comes from x
// in 32 bits; 216 ln 2 is off by 2^-46 with ln 2 in 64.
__device__ __forceinline__ double exp_f64(double x, float x32) {
  const float n = __builtin_rintf(x32 * 1.44269504f);
  const double r = __builtin_fma((double)n, -0.6931471805599453, x);
  double p = 1.0 / 362880;
  p = __builtin_fma(p, r, 1.0 / 40320);
  p = __builtin_fma(p, r, 1.0 / 5040);
  p = __builtin_fma(p, r, 1.0 / 720);
  p = __builtin_fma(p, r, 1.0 / 120);
  p = __builtin_fma(p, r, 1.0 / 24);
  p = __builtin_fma(p, r, 1.0 / 6);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_amdgcn_ldexp(p, (int)n);
}
// 1 / d of a normal d: the hardware's estimate (2^-24 at the least) and a step of Newton's iteration
__device__ __forceinline__ double rcp_f64(double d) {
  const double y = __builtin_amdgcn_rcp(d);
  return __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
}

// score[v] in 64 bits, rounded once; 0 for masked experts (all of a token masked: all 0).
// Two scores that float32 arithmetic would exchange, or make equal, change which expert
// a token takes or their order: with a float32 exponential one token in about 40,000
// (256 experts in 8 groups, top 8).  Here the sum of errors is 2^-11 of a rounding, and
// of such tokens one in 2000 remains.
template <int V>
__device__ __forceinline__ void exact_scores(const float* z, bool softmax, float* score) {
  if (!softmax) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float z32 = fmaxf(-fabsf(z[v]), -150.0f);         // below it a float32 score is 0 or 1
      const double x = exp_f64((double)z32, z32);
      score[v] = (float)((z[v] < 0.0f ? x : 1.0) * rcp_f64(1.0 + x));
    }
    return;
  }
  float top = z[0];
#pragma unroll
  for (int v = 1; v < V; ++v) top = fmaxf(top, z[v]);
  top = wave_max(top);
  double e[V], sum = 0.0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float z32 = z[v] - top;
    e[v] = z[v] == top ? 1.0 : z32 > -150.0f ? exp_f64((double)z[v] - (double)top, z32) : 0.0;
    e[v] = z[v] == minus_inf() ? 0.0 : e[v];
    sum += e[v];
  }
  sum = wave_sum_f64(sum);
  const double by = sum > 0.0 ? rcp_f64(sum) : 0.0;
#pragma unroll
  for (int v = 0; v < V; ++v) score[v] = (float)(e[v] * by);
}

// e^-|z|, of which the sigmoid is made: scores go down to float32's smallest numbers
__device__ __forceinline__ float sigmoid_of(float z, float x) {
  return (z < 0.0f ? x : 1.0f) * __builtin_amdgcn_rcpf(1.0f + x);
}

// score[v] in float32, and the sum of all of them (1 for a softmax, 0 where all are masked);
// of a sigmoid also x[v] = e^-|z[v]|.
template <int V>
__device__ __forceinline__ float scores(const float* z, bool softmax, float* score, float* x) {
  float sum = 0.0f;
  if (!softmax) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = exp_f32(-fabsf(z[v]));
      score[v] = sigmoid_of(z[v], x[v]);
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
    score[v] = z[v] == minus_inf() ? 0.0f : z[v] == top ? 1.0f : exp_f32(z[v] - top);
    sum += score[v];
  }
  sum = wave_sum(sum);
  const float by = sum > 0.0f ? __builtin_amdgcn_rcpf(sum) : 0.0f;   // of at least 1
#pragma unroll
  for (int v = 0; v < V; ++v) score[v] *= by;
  return sum > 0.0f ? 1.0f : 0.0f;
}

// score[v] over their sum; a softmax's are that already.
template <int V>
__device__ __forceinline__ void shares(float* score, float sum, bool softmax) {
  if (softmax) return;
  // 1 / sum is infinite for the sum of the smallest scores: those are taken times 2^64 before it
  const bool tiny = sum < 1e-30f;
  const float up = tiny ? 18446744073709551616.0f : 1.0f;
  const float by = sum > 0.0f ? __builtin_amdgcn_rcpf(sum * up) : 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) score[v] = score[v] * up * by;
}

// Sequence s's tokens [a, b), inside [0, T); T < 2^24
__device__ __forceinline__ void bounds_of(const int32_t* cu, int s, int T, int* a, int* b) {
  *a = cu ? min(max(cu[s], 0), T) : 0;
  *b = cu ? max(min(max(cu[s + 1], 0), T), *a) : T;
}

// The last of S sequences that starts at token t or before, 0 if none does, by the
// wave's 64 probes at a time.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int S, int t, int lane) {
  int lo = 0;
  while (S > 1) {
    const int step = (S + 63) / 64, at = lane * step;
    const int before = __popcll(__ballot(at < S && cu[lo + min(at, S - 1)] <= t));
    const int skip = max(before - 1, 0) * step;
    lo += skip;
    S = min(step, S - skip);
  }
  return lo;
}

// The two largest of two disjoint sets, each given by its two largest
__device__ __forceinline__ void join_two(uint32_t& a, uint32_t& b, uint32_t c, uint32_t d) {
  b = max(min(a, c), max(b, d));
  a = max(a, c);
}
template <int CTRL>
__device__ __forceinline__ void join_dpp(uint32_t& a, uint32_t& b) {
  join_two(a, b, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, CTRL, 0xF, 0xF, true),
           (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, CTRL, 0xF, 0xF, true));
}

}  // namespace

// ----------------------------------------------------------------------------
// gate
// ----------------------------------------------------------------------------
template <int V, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void moe_gate_kernel(const MoeGate p) {
  __shared__ uint32_t slots[kWaves][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * kWaves + wave));
  if (t >= p.T) return;                                       // waves work apart: no barrier follows
  const int E = (int)p.E, G = (int)p.groups;
  float z[V], top_z = 0.0f, all = 0.0f;
  load_logits<V, VEC>(p.logits, p.f32, t * p.ld, E, lane, z);
  uint32_t key[V];
  if (p.bias) {
    uint32_t b[V];
    if (VEC && p.bias_wide) load_words<V, true>((const uint32_t*)p.bias, lane * V, E, 0, b);
    else load_words<V, false>((const uint32_t*)p.bias, lane * V, E, 0, b);
    float score[V];
    exact_scores<V>(z, p.softmax, score);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float k = score[v] + bits_f32(b[v]);
      key[v] = z[v] > minus_inf() && k > minus_inf() ? order_of(k) : 0;
      slots[wave][lane * V + v] = f32_bits(score[v]);
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = z[v] > minus_inf() ? order_of(z[v]) : 0;
    if (p.softmax) {
      top_z = z[0];
#pragma unroll
      for (int v = 1; v < V; ++v) top_z = fmaxf(top_z, z[v]);
      top_z = wave_max(top_z);
#pragma unroll
      for (int v = 0; v < V; ++v) all += z[v] == minus_inf() ? 0.0f : z[v] == top_z ? 1.0f : exp_f32(z[v] - top_z);
      all = wave_sum(all);
    }
  }
  if (G > 1) {
    const int size = E / G, lanes = size / V;                 // a group's lanes, where it has whole ones
    uint32_t a = 0, b = 0;                                    // the two largest keys of the lane's group
    if (size % V == 0 && (lanes & (lanes - 1)) == 0) {
      a = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) join_two(a, b, key[v], 0);
      // over 2, 4, 8, 16 lanes: those of a set already joined hold the same, so a mirror
      // of a row's half, or of the row, brings the other half's
      if (lanes >= 2) join_dpp<0xB1>(a, b);                   // quad_perm 1,0,3,2
      if (lanes >= 4) join_dpp<0x4E>(a, b);                   // quad_perm 2,3,0,1
      if (lanes >= 8) join_dpp<0x141>(a, b);                  // row_half_mirror
      if (lanes >= 16) join_dpp<0x140>(a, b);                 // row_mirror
      if (lanes >= 32) join_two(a, b, (uint32_t)__shfl_xor((int)a, 16), (uint32_t)__shfl_xor((int)b, 16));
      const uint32_t value = p.bias && b ? order_of(float_of(a) + float_of(b)) : a;
      const int mine = lane / lanes;
      int before = 0;                                         // groups that come before the lane's
      for (int g = 0; g < G; ++g) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)value, g * lanes);
        before += o > value || (o == value && g < mine);
      }
      if (before >= (int)p.keep) {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = 0;
      }
    } else {
      // any size: keys through LDS, lane g looks at group g
      __shared__ uint32_t keys[kWaves][64 * V];
#pragma unroll
      for (int v = 0; v < V; ++v) keys[wave][lane * V + v] = key[v];
      __threadfence_block();
      __builtin_amdgcn_wave_barrier();
      if (lane < G)
        for (int i = 0; i < size; ++i) join_two(a, b, keys[wave][lane * size + i], 0);
      const uint32_t value = p.bias && b ? order_of(float_of(a) + float_of(b)) : a;
      int before = 0;
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
  }
  int id = -1;
  uint32_t mine = 0;
  for (int k = 0; k < (int)p.topk; ++k) {
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max(best, key[v]);
    const uint32_t top = wave_max_uniform(best);
    if (top == 0) break;                                      // no expert is left
    const int who = __ffsll((unsigned long long)__ballot(best == top)) - 1;
    int at = V - 1;
#pragma unroll
    for (int v = V - 2; v >= 0; --v)
      if (key[v] == top) at = v;
    const int e = who * V + __builtin_amdgcn_readlane(at, who);
    if (lane == k) id = e, mine = top;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane * V + v == e) key[v] = 0;
  }
  // lane k: the score of the token's k-th expert
  float w = 0.0f;
  if (p.bias) {
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
    if (id >= 0) w = bits_f32(slots[wave][id]);
  } else if (id >= 0) {
    const float zk = float_of(mine);
    if (!p.softmax) w = sigmoid_of(zk, exp_f32(-fabsf(zk)));
    else w = (zk == top_z ? 1.0f : exp_f32(zk - top_z)) * __fdiv_rn(1.0f, all);
  }
  if (p.normalize) {
    const float sum = wave_sum(w);
    w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
  }
  if (lane < (int)p.topk) {
    p.indices[t * (int)p.topk + lane] = id;                   // T * topk < 2^31
    p.weights[t * (int)p.topk + lane] = w * p.route_scale;
  }
}

namespace {

// Calls CALL(V, VEC) with V registers a lane for E experts; VEC where rows are read V logits at a time.
#define FP8BS_BY_EXPERTS(p, CALL)                                                   \
  {                                                                                 \
    const int V = experts_a_lane((p).E);                                            \
    const bool vec = wide_rows((p).logits, (p).ld, (p).E, V, (p).f32);              \
    if (V == 1) { CALL(1, false); }                                                 \
    else if (V == 2) { if (vec) { CALL(2, true); } else { CALL(2, false); } }       \
    else if (V == 4) { if (vec) { CALL(4, true); } else { CALL(4, false); } }       \
    else if (V == 8) { if (vec) { CALL(8, true); } else { CALL(8, false); } }       \
    else { if (vec) { CALL(16, true); } else { CALL(16, false); } }                 \
  }
int experts_a_lane(int64_t E) { return E <= 64 ? 1 : E <= 128 ? 2 : E <= 256 ? 4 : E <= 512 ? 8 : 16; }
bool wide_rows(const void* p, int64_t ld, int64_t E, int V, bool f32) {
  const int wide = std::min(V * (f32 ? 4 : 2), 16);
  return V > 1 && E % V == 0 && ld % V == 0 && (uintptr_t)p % wide == 0;
}

}  // namespace

hipError_t launch_moe_gate(const MoeGate& q, hipStream_t stream) {
  MoeGate p = q;
  p.bias_wide = (uintptr_t)p.bias % 16 == 0;
  const dim3 grid((unsigned)((p.T + kWaves - 1) / kWaves)), block(64 * kWaves);
#define CALL(V, VEC) moe_gate_kernel<V, VEC><<<grid, block, 0, stream>>>(p)
  FP8BS_BY_EXPERTS(p, CALL)
#undef CALL
  return hipGetLastError();
}

// ----------------------------------------------------------------------------
// balance.  Workgroup b takes tokens [b*R, (b+1)*R), whatever the sequences'
// lengths; of each sequence that has some of them it leaves the sums of shares and
// the counts in slot b + s of the workspace (b + s grows by one from a workgroup's
// sequence to the next one's, so no two share a slot).  The second kernel adds a
// sequence's slots up, which lie next to each other, in order, and makes its loss.
// ----------------------------------------------------------------------------
namespace {

constexpr int kBalanceWaves = 8;
constexpr int kBalanceRows = 16;     // tokens of a workgroup: two a wave
constexpr int kBalanceGroups = 512;  // more workgroups than this take more tokens each

struct BalancePlan {
  int64_t rows, groups, width;       // tokens a workgroup, workgroups, floats of a slot
};
BalancePlan balance_plan(int64_t T, int64_t E) {
  const int64_t least = (T + kBalanceGroups - 1) / kBalanceGroups;
  const int64_t rows = std::max<int64_t>(kBalanceRows, (least + kBalanceWaves - 1) / kBalanceWaves * kBalanceWaves);
  return {rows, (T + rows - 1) / rows, (E + 3) / 4 * 4};
}

// A sequence's results from its sums, by one workgroup: probs, counts, and the loss
// E / (topk * n) * sum counts * probs.  get(e, &shares, &hits); `red` one float a wave.
template <typename F>
__device__ __forceinline__ void finish_sequence(const MoeBalance& p, int s, int n, float* red, F get) {
  const int E = (int)p.E;
  const float mean = n > 0 ? __fdiv_rn(1.0f, (float)n) : 0.0f;
  float part = 0.0f;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float q;
    int32_t h;
    get(e, &q, &h);
    q *= mean;
    p.probs[(int64_t)s * E + e] = q;
    p.counts[(int64_t)s * E + e] = h;
    part = __builtin_fmaf(q, (float)h, part);
  }
  part = wave_sum(part);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    part = 0.0f;
    for (int w = 0; w < (int)blockDim.x / 64; ++w) part += red[w];
    p.loss[s] = n > 0 ? part * __fdiv_rn((float)E, (float)p.topk * (float)n) : 0.0f;
  }
  __syncthreads();
}

}  // namespace

// ONE: a workgroup a sequence, which makes its results itself.
template <int V, bool VEC, bool ONE>
__global__ __launch_bounds__(64 * kBalanceWaves) void moe_balance_kernel(const MoeBalance p, int rows, int width) {
  __shared__ float sums[kBalanceWaves][64 * V];
  __shared__ int32_t hits[64 * V];
  __shared__ float red[kBalanceWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = (int)p.E;
  const int lo = ONE ? 0 : (int)blockIdx.x * rows, hi = ONE ? (int)p.T : min(lo + rows, (int)p.T);
  int s = ONE ? (int)blockIdx.x : p.cu ? __builtin_amdgcn_readfirstlane(sequence_of(p.cu, (int)p.S, lo, lane)) : 0;
  int empty = 0;                                              // sequences without a token, one after another
  for (; s < (int)p.S; ++s) {
    int a, b;
    bounds_of(p.cu, s, (int)p.T, &a, &b);
    if (!ONE && a >= hi) break;
    const int n = b - a;
    a = max(a, lo);
    b = min(b, hi);
    if (!ONE && a >= b) {
      // the third empty one on: to the sequence that has token a, past all that are empty (100000 of them between the
      // tokens of a workgroup 0.43 ms, one by one 12.8; where one in two is empty the search costs more than a step)
      if (++empty > 2) s = max(s, __builtin_amdgcn_readfirstlane(sequence_of(p.cu, (int)p.S, a, lane)) - 1);
      continue;
    }
    empty = 0;
    for (int i = threadIdx.x; i < 64 * V; i += 64 * kBalanceWaves) hits[i] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
    for (int t = a + wave; t < b; t += kBalanceWaves) {
      const int32_t id = lane < (int)p.topk ? p.indices[t * (int)p.topk + lane] : -1;
      float z[V], score[V], x[V];
      load_logits<V, VEC>(p.logits, p.f32, t * p.ld, E, lane, z);
      const float sum = scores<V>(z, p.softmax, score, x);
      shares<V>(score, sum, p.softmax);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += score[v];
      if (id >= 0 && id < E) atomicAdd(&hits[id], 1);         // whole numbers: any order gives the same
    }
#pragma unroll
    for (int v = 0; v < V; ++v) sums[wave][lane * V + v] = acc[v];
    __syncthreads();
    const auto get = [&](int e, float* q, int32_t* h) {
      *q = 0.0f;
#pragma unroll
      for (int w = 0; w < kBalanceWaves; ++w) *q += sums[w][e];
      *h = hits[e];
    };
    if (ONE) {
      finish_sequence(p, s, n, red, get);
      return;
    } else {
      const int64_t slot = (int64_t)((int)blockIdx.x + s) * width;
      for (int e = threadIdx.x; e < width; e += 64 * kBalanceWaves) {
        float q = 0.0f;
        int32_t h = 0;
        if (e < E) get(e, &q, &h);
        p.part_probs[slot + e] = q;
        p.part_counts[slot + e] = h;
      }
      __syncthreads();
    }
  }
}

constexpr int kJoinThreads = 1024, kJoinGroups = 32;
__global__ __launch_bounds__(kJoinThreads) void moe_balance_join_kernel(const MoeBalance p, int rows, int width) {
  __shared__ float4 sums[kJoinThreads];
  __shared__ int4 hits[kJoinThreads];
  __shared__ float red[kJoinThreads / 64];
  const int s = blockIdx.x;
  int a, b;
  bounds_of(p.cu, s, (int)p.T, &a, &b);
  const int first = a / rows, last = b > a ? (b - 1) / rows + 1 : first;       // workgroups with some of its tokens
  // a thread adds up 4 experts of every `groups`-th slot, 4 slots' loads at a time
  const int cols = width / 4, groups = min(kJoinThreads / cols, kJoinGroups);
  const int grp = (int)threadIdx.x / cols, col = (int)threadIdx.x - grp * cols;
  float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  int4 h = make_int4(0, 0, 0, 0);
  if (grp < groups) {
    for (int g = first + grp; g < last; g += 4 * groups) {
      float4 x[4];
      int4 y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = (int64_t)(min(g + i * groups, last - 1) + s) * width;
        x[i] = ((const float4*)(p.part_probs + at))[col];
        y[i] = ((const int4*)(p.part_counts + at))[col];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (g + i * groups >= last) break;
        q.x += x[i].x, q.y += x[i].y, q.z += x[i].z, q.w += x[i].w;
        h.x += y[i].x, h.y += y[i].y, h.z += y[i].z, h.w += y[i].w;
      }
    }
    sums[grp * cols + col] = q;
    hits[grp * cols + col] = h;
  }
  __syncthreads();
  finish_sequence(p, s, b - a, red, [&](int e, float* q, int32_t* h) {
    *q = 0.0f;
    *h = 0;
#pragma unroll 4
    for (int g = 0; g < groups; ++g) {
      *q += ((const float*)sums)[g * width + e];
      *h += ((const int32_t*)hits)[g * width + e];
    }
  });
}

// A workgroup a sequence, and no second kernel, where that has few tokens to go through: 16 tokens of 256 experts 7.6 us
// (with the gradient) where two kernels take 9.9; 64 tokens of one sequence 10.7 and 10.4, of eight 8.2 and 14.1.
constexpr int kBalanceAtOnce = 32;
static bool balance_at_once(int64_t T) { return T <= kBalanceAtOnce; }

int64_t moe_balance_workspace_bytes(int64_t T, int64_t S, int64_t E) {
  const BalancePlan plan = balance_plan(T, E);
  return balance_at_once(T) ? 0 : 8 * (plan.groups + S) * plan.width;
}

hipError_t launch_moe_balance(const MoeBalance& q, hipStream_t stream) {
  MoeBalance p = q;
  const BalancePlan plan = balance_plan(p.T, p.E);
  const bool one = balance_at_once(p.T);
  p.part_probs = (float*)p.workspace;
  p.part_counts = (int32_t*)p.workspace + (plan.groups + p.S) * plan.width;
  const dim3 grid((unsigned)(one ? p.S : plan.groups)), block(64 * kBalanceWaves);
#define CALL(V, VEC)                                                                                        \
  if (one) moe_balance_kernel<V, VEC, true><<<grid, block, 0, stream>>>(p, (int)plan.rows, (int)plan.width);          \
  else moe_balance_kernel<V, VEC, false><<<grid, block, 0, stream>>>(p, (int)plan.rows, (int)plan.width)
  FP8BS_BY_EXPERTS(p, CALL)
#undef CALL
  if (!one) moe_balance_join_kernel<<<dim3((unsigned)p.S), dim3(kJoinThreads), 0, stream>>>(p, (int)plan.rows, (int)plan.width);
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
template <int V, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void moe_gate_bwd_kernel(const MoeGateBwd p) {
  __shared__ float slots[kWaves][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * kWaves + wave));
  if (t >= p.T) return;
  const int E = (int)p.E, K = (int)p.topk;
  int e = -1;
  float uk = 0.0f;
  if (p.d_weights && lane < K) {
    e = p.indices[t * K + lane];                              // T * topk < 2^31
    uk = p.d_weights[t * K + lane];
    if (e < 0 || e >= E) e = -1, uk = 0.0f;
  }
  float z[V], score[V], x[V], u[V];
  load_logits<V, VEC>(p.logits, p.f32, t * p.ld, E, lane, z);
  // the token's sequence, asked for before the scores are made
  int a = 0, b = 0;
  uint32_t hits[V];
  float dl = 0.0f;
  if (p.d_loss) {
    const int s = p.cu ? sequence_of(p.cu, (int)p.S, t, lane) : 0;
    bounds_of(p.cu, s, (int)p.T, &a, &b);
    load_words<V, false>((const uint32_t*)p.counts + (int64_t)s * E, lane * V, E, 0, hits);
    dl = p.d_loss[s];
  }
  const float sum = scores<V>(z, p.softmax, score, x);
#pragma unroll
  for (int v = 0; v < V; ++v) u[v] = 0.0f;
  if (p.d_loss && t >= a && t < b) {
    const float n = (float)(b - a);
    const float c = dl * (float)E * __builtin_amdgcn_rcpf((float)K * n) * __builtin_amdgcn_rcpf(n);
    float share[V], mean = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) share[v] = score[v];
    shares<V>(share, sum, p.softmax);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      u[v] = c * (float)(int32_t)hits[v];
      mean = __builtin_fmaf(u[v], share[v], mean);
    }
    mean = wave_sum(mean);
#pragma unroll
    for (int v = 0; v < V; ++v) u[v] = (u[v] - mean) * share[v];
  }
  if (p.d_weights) {
    // lane k: the score of the token's k-th expert
#pragma unroll
    for (int v = 0; v < V; ++v) slots[wave][lane * V + v] = score[v];
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
    float own = e >= 0 ? slots[wave][e] : 0.0f;
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
      for (int v = 0; v < V; ++v) u[v] += ek == lane * V + v ? add : 0.0f;
    }
  }
  float all = 0.0f;
  if (p.softmax) {
#pragma unroll
    for (int v = 0; v < V; ++v) all += u[v];
    all = wave_sum(all);
  }
  float dz[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (p.softmax) {
      dz[v] = __builtin_fmaf(-score[v], all, u[v]);
    } else {
      dz[v] = u[v] * sigmoid_of(-z[v], x[v]);                 // 1 - score without the cancellation near 1
    }
  }
  const int64_t at = (int64_t)t * E + lane * V;
  if (VEC) {
    if (lane * V >= E) return;
    if (p.out_f32) {
      if (V >= 4) {
#pragma unroll
        for (int v = 0; v < V; v += 4)
          *(float4*)((float*)p.d_logits + at + v) = make_float4(dz[v], dz[(v + 1) % V], dz[(v + 2) % V], dz[(v + 3) % V]);
      } else {
        *(float2*)((float*)p.d_logits + at) = make_float2(dz[0], dz[1 % V]);
      }
    } else {
      if (V >= 4) {
#pragma unroll
        for (int v = 0; v < V; v += 4)
          *(uint2*)((uint16_t*)p.d_logits + at + v) =
              make_uint2(pack2_bf16(dz[v], dz[(v + 1) % V]), pack2_bf16(dz[(v + 2) % V], dz[(v + 3) % V]));
      } else {
        *(uint32_t*)((uint16_t*)p.d_logits + at) = pack2_bf16(dz[0], dz[1 % V]);
      }
    }
    return;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (lane * V + v >= E) continue;
    if (p.out_f32) ((float*)p.d_logits)[at + v] = dz[v];
    else ((uint16_t*)p.d_logits)[at + v] = (uint16_t)pack2_bf16(dz[v], 0.0f);
  }
}

hipError_t launch_moe_gate_bwd(const MoeGateBwd& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + kWaves - 1) / kWaves)), block(64 * kWaves);
#define CALL(V, VEC) moe_gate_bwd_kernel<V, VEC><<<grid, block, 0, stream>>>(p)
  FP8BS_BY_EXPERTS(p, CALL)
#undef CALL
  return hipGetLastError();
}

}  // namespace fp8bs
