// swiglu.hip -- the activation between the two products of an expert,
//   a = g * sigmoid(g) * u,
// with block-scaled FP8 output for the second product (act_quant's rule:
// "DeepSeek-V3 Administrator & Developer Guide" 8.5.1) or bf16, and its gradient.
// HBM-bound: every element is read and written once; 16 consecutive lanes hold a
// block of 128.  32768 x 2048 to codes 56.1 us (338 MB, 6.0 TB/s), the gradient of
// 29999 x 2048 95.5 us (614 MB, 6.4 TB/s).  It was bound by instructions (87 us) with the
// library's exponential and correctly rounded quotients, 48 a value; it takes 23.
#include "device_common.h"
#include "launch.h"

namespace fp8bs {

namespace {

constexpr int kThreads = 256;
// Rows that a thread takes where there are many.  us with 2 / 3 / 4 / 8: 32768 x 2048 55.9 / 56.1 / 58.0 / 58.8, a buffer
// of them of which a count says that 2000 are there 7.0 / 5.7 / 5.5 / 7.0; gradient of 29999 x 2048 with 2 / 4: 95.5 / 98.4.
constexpr int kPasses = 3, kBwdPasses = 2;

// A workgroup's 256 threads are R = 256 / C rows of C vectors, C the largest power of
// two, up to 256, that divides a row's vectors: no lane is idle and a thread's row and
// column cost shifts.  C >= 16, so 16 lanes hold a block of 128.
struct Tile {
  int64_t row;         // a thread's first row; the next ones lie `step` apart
  uint32_t col;        // its vector in them
  int step;
};
__device__ __forceinline__ Tile tile_of(int shift, uint32_t chunks, int passes) {
  const uint32_t band = blockIdx.x / chunks, chunk = blockIdx.x - band * chunks;
  const int step = kThreads >> shift;
  return {(int64_t)band * (step * passes) + (threadIdx.x >> shift),
          (chunk << shift) + (threadIdx.x & ((1u << shift) - 1)), step};
}

// Below -80 a gate's sigmoid is e^g to float32's last bit, and soon outside its normal range, while g * e^g * u need not
// be.  Such values are made in two factors h = e^(g / 2), in range down to -174.  They are rare: a wave without any
// passes them by with a maximum and a branch.  (All values in two factors: 28 instructions a value for 23.)
constexpr float kDeep = -80.0f;
__device__ __forceinline__ bool any_deep(const float* g) {
  uint32_t most = f32_bits(g[0]);                            // of negative floats the largest magnitude, above all others
#pragma unroll
  for (int i = 1; i < 8; ++i) most = max(most, f32_bits(g[i]));
  return __any(most > f32_bits(kDeep));
}

// rows that the call has: all, or fewer by the device's count
__device__ __forceinline__ int64_t rows_of(const int32_t* n_rows, int64_t M) {
  return n_rows ? min(max<int64_t>(*n_rows, 0), M) : M;
}

template <bool NT>
__device__ __forceinline__ uint4 load_row(const void* p, int64_t row, int64_t ld, uint32_t col) {
  const uint4* at = (const uint4*)((const uint16_t*)p + row * ld) + col;
  return NT ? load_nt(at) : *at;
}

}  // namespace

template <int PASSES, bool NT>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(const SwiGlu p, int shift, uint32_t chunks) {
  const Tile t = tile_of(shift, chunks, PASSES);
  const int64_t nv = p.N / 8, rows = rows_of(p.n_rows, p.M);
  if (t.row >= rows) return;                                 // 16 lanes together, as below
  uint4 g[PASSES], u[PASSES];
#pragma unroll
  for (int k = 0; k < PASSES; ++k) {
    const int64_t r = t.row + k * t.step < rows ? t.row + k * t.step : t.row;
    g[k] = load_row<NT>(p.gate, r, p.ld_g, t.col);
    u[k] = load_row<NT>(p.up, r, p.ld_u, t.col);
  }
#pragma unroll
  for (int k = 0; k < PASSES; ++k) {
    const int64_t r = t.row + k * t.step;
    if (r >= rows) return;
    float x[8], b[8], a[8];
    unpack8(g[k], x);
    unpack8(u[k], b);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = x[i] * sigmoid_f32(x[i]) * b[i];
    if (any_deep(x)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = exp_f32(0.5f * x[i]);
        if (x[i] < kDeep) a[i] = x[i] * h * (b[i] * h);
      }
    }
    const int64_t at = r * nv + t.col;
    if (p.y) store_nt((uint4*)p.y + at, pack8(a));
    if (p.q) {
      float sc;
      store_nt((uint2*)p.q + at, quant8(a, p.ue8m0, &sc));
      if ((threadIdx.x & 15) == 0) p.s[at / 16] = sc;
    }
  }
}

// du = dy * g * sigmoid(g),  dg = dy * u * sigmoid(g) * (1 + g * (1 - sigmoid(g)))
template <int PASSES, bool NT>
__global__ __launch_bounds__(kThreads) void swiglu_bwd_kernel(const SwiGluBwd p, int shift, uint32_t chunks) {
  const Tile t = tile_of(shift, chunks, PASSES);
  const int64_t rows = rows_of(p.n_rows, p.M);
  if (t.row >= rows) return;
  uint4 g[PASSES], u[PASSES], d[PASSES];
#pragma unroll
  for (int k = 0; k < PASSES; ++k) {
    const int64_t r = t.row + k * t.step < rows ? t.row + k * t.step : t.row;
    g[k] = load_row<NT>(p.gate, r, p.ld_g, t.col);
    u[k] = load_row<NT>(p.up, r, p.ld_u, t.col);
    d[k] = load_row<NT>(p.dy, r, p.N, t.col);
  }
#pragma unroll
  for (int k = 0; k < PASSES; ++k) {
    const int64_t r = t.row + k * t.step;
    if (r >= rows) return;
    float a[8], b[8], e[8], dg[8], du[8];
    unpack8(g[k], a);
    unpack8(u[k], b);
    unpack8(d[k], e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid_f32(a[i]), x = e[i] * s;
      dg[i] = x * b[i] * __builtin_fmaf(a[i], 1.0f - s, 1.0f);
      du[i] = x * a[i];
    }
    if (any_deep(a)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = exp_f32(0.5f * a[i]), x = e[i] * h;
        if (a[i] < kDeep) dg[i] = x * (b[i] * h) * (1.0f + a[i]), du[i] = x * (a[i] * h);
      }
    }
    store_nt((uint4*)((uint16_t*)p.dgate + r * p.ld_dg) + t.col, pack8(dg));
    store_nt((uint4*)((uint16_t*)p.dup + r * p.ld_du) + t.col, pack8(du));
  }
}

namespace {

struct Plan {
  int shift;
  uint32_t chunks;
  int passes;
  int64_t grid;
};
// One row a thread while that leaves no more than 8 workgroups a CU, so that few rows
// are spread over the card.
Plan plan_of(int64_t M, int64_t N, int most) {
  const int64_t nv = N / 8;
  int shift = 4;
  while (shift < 8 && nv % (2 << shift) == 0) ++shift;
  const int64_t chunks = nv >> shift, step = kThreads >> shift;
  const int64_t one = (M + step - 1) / step;
  const int passes = one <= 2048 / chunks ? 1 : most;
  return {shift, (uint32_t)chunks, passes, (one + passes - 1) / passes * chunks};
}

}  // namespace

// One launch: at most 2^32 - 1 threads.
bool swiglu_fits(int64_t M, int64_t N) {
  if (M <= 0 || N <= 0) return true;
  if (N >= (int64_t)1 << 31 || M >= (int64_t)1 << 40) return false;
  const Plan q = plan_of(M, N, kBwdPasses);
  return q.grid / q.chunks <= (((int64_t)1 << 32) - 1) / kThreads / q.chunks;
}

hipError_t launch_swiglu(const SwiGlu& p, hipStream_t stream) {
  const Plan q = plan_of(p.M, p.N, kPasses);
  const int64_t bytes = p.M * p.N * (4 + (p.y ? 2 : 0) + (p.q ? 1 : 0));
  const auto kernel = q.passes == 1 ? swiglu_kernel<1, false>
                      : bytes >= kHintBytes ? swiglu_kernel<kPasses, true> : swiglu_kernel<kPasses, false>;
  kernel<<<dim3((unsigned)q.grid), dim3(kThreads), 0, stream>>>(p, q.shift, q.chunks);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const SwiGluBwd& p, hipStream_t stream) {
  const Plan q = plan_of(p.M, p.N, kBwdPasses);
  const auto kernel = q.passes == 1 ? swiglu_bwd_kernel<1, false>
                      : 10 * p.M * p.N >= kHintBytes ? swiglu_bwd_kernel<kBwdPasses, true>
                                                       : swiglu_bwd_kernel<kBwdPasses, false>;
  kernel<<<dim3((unsigned)q.grid), dim3(kThreads), 0, stream>>>(p, q.shift, q.chunks);
  return hipGetLastError();
}

}  // namespace fp8bs
