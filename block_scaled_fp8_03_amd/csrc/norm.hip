// norm.hip -- RMSNorm with the residual's addition and block-scaled FP8 output,
// and its gradient (the norms of the pages' blocks: "DeepSeek-V3 Administrator &
// Developer Guide" 1.1, in front of the FP8 linears of 6.3).
//
//   t = x + res,  c = t / sqrt(mean(t^2) + eps) * w,
//   res_out = round(t), y = bf16(c), per 128: s = act_quant's rule on c, q = e4m3(c / s)
//
// HBM-bound: a row is read once, held in registers while its squares are summed,
// and written once.  One vector of 8 a lane up to 8192 columns, that is a row spread
// over as many waves as it has 512 columns: 1 x 7168 3.07 us (two vectors a lane 3.29,
// four 4.0), 4096 x 7168 46.1 (46.3, 47.8).  4096 x 7168 with a bf16 residual, codes and
// bf16 out move 265 MB at 5.7 TB/s.
#include <algorithm>

#include "device_common.h"
#include "launch.h"

namespace fp8bs {

namespace {

constexpr int kThreads = 256;        // of a workgroup with several rows
constexpr int kMaxThreads = 1024;    // of a workgroup with one
constexpr int kMaxK = 32768;

// Sum over the TPR lanes of a row (TPR 16, 32, 64: inside a wave; 0: the workgroup,
// through `red`, one float a wave).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  if (TPR == 16) return row16_sum(v);
  if (TPR == 32) {
    v = row16_sum(v);
    return v + __shfl_xor(v, 16);
  }
  v = wave_sum(v);
  if (TPR == 64) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float sum = 0.0f;
  for (int i = 0; i < (int)blockDim.x / 64; ++i) sum += red[i];
  return sum;
}

// 8 elements of a row as floats
template <bool F32>
__device__ __forceinline__ void floats_of(const uint4* u, float* f) {
  if (F32) {
    const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = bits_f32(w[i]);
  } else {
    unpack8(u[0], f);
  }
}
// NT: read once (the norm's weight is read by every row)
template <bool F32, bool NT>
__device__ __forceinline__ void load8(const void* p, int64_t v, float* f) {
  uint4 u[F32 ? 2 : 1];
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) {
    const uint4* at = (const uint4*)p + (F32 ? 2 * v + i : v);
    u[i] = NT ? load_nt(at) : *at;
  }
  floats_of<F32>(u, f);
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t v, const float* f) {
  if (F32) {
    store_nt((uint4*)p + 2 * v, make_uint4(f32_bits(f[0]), f32_bits(f[1]), f32_bits(f[2]), f32_bits(f[3])));
    store_nt((uint4*)p + 2 * v + 1, make_uint4(f32_bits(f[4]), f32_bits(f[5]), f32_bits(f[6]), f32_bits(f[7])));
  } else {
    store_nt((uint4*)p + v, pack8(f));
  }
}
__device__ __forceinline__ void load_w(const RmsNorm& p, int64_t v, float* f) {
  if (p.w_f32) load8<true, false>(p.w, v, f);
  else load8<false, false>(p.w, v, f);
}

}  // namespace

// ----------------------------------------------------------------------------
// forward: TPR lanes a row (0: the workgroup), VPL vectors of 8 a lane; RES 0
// none, 1 bf16, 2 float32.  16 consecutive lanes hold a block of 128.
// ----------------------------------------------------------------------------
template <int TPR, int VPL, int RES, bool NT>
__global__ __launch_bounds__(TPR ? kThreads : kMaxThreads) void rmsnorm_kernel(const RmsNorm p) {
  __shared__ float red[kMaxThreads / 64];
  const int tpr = TPR ? TPR : (int)blockDim.x;
  const int lane = TPR ? (int)threadIdx.x % TPR : (int)threadIdx.x;
  const int64_t m = TPR ? (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR : (int64_t)blockIdx.x;
  const int64_t mm = TPR ? min(m, p.M - 1) : m;              // a row to read from where there is none
  const int nv = (int)(p.K / 8);
  const uint4* xr = (const uint4*)((const uint16_t*)p.x + mm * p.ld_x);
  float t[VPL][8];
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int v = lane + j * tpr, vv = min(v, nv - 1);
    unpack8(NT ? load_nt(xr + vv) : xr[vv], t[j]);
    if (RES) {
      float r[8];
      load8<RES == 2, NT>(p.res, mm * nv + vv, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[j][i] += r[i];
    }
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = __builtin_fmaf(t[j][i], t[j][i], a);
    sum += v < nv ? a : 0.0f;
  }
  sum = row_sum<TPR>(sum, red);
  const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(sum, (float)p.K) + p.eps));
  if (TPR && m >= p.M) return;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int v = lane + j * tpr;
    if (v >= nv) break;                                      // whole blocks of 128: nv is a multiple of 16
    const int64_t at = m * nv + v;
    if (RES) store8<RES == 2>(p.res_out, at, t[j]);
    float c[8];
    load_w(p, v, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = t[j][i] * r * c[i];
    if (p.y) store_nt((uint4*)p.y + at, pack8(c));
    if (p.q) {
      float sc;
      store_nt((uint2*)p.q + at, quant8(c, p.ue8m0, &sc));
      if ((lane & 15) == 0) p.s[at / 16] = sc;
    }
  }
}

namespace {

// Lanes a row (16, 32, 64 inside a wave; else the threads of its workgroup) and vectors a lane.
struct RowPlan {
  int tpr, vpl;
};
RowPlan plan_of(int64_t K) {
  const int64_t nv = K / 8;
  if (nv <= 64) return {nv <= 16 ? 16 : nv <= 32 ? 32 : 64, 1};
  const int vpl = nv <= kMaxThreads ? 1 : nv <= 2 * kMaxThreads ? 2 : 4;
  return {(int)((nv + 64 * vpl - 1) / (64 * vpl)) * 64, vpl};
}

template <int RES, bool NT>
void launch_fwd(const RmsNorm& p, hipStream_t stream) {
  const RowPlan plan = plan_of(p.K);
  const int rows = plan.tpr <= 64 ? kThreads / plan.tpr : 1;
  const dim3 grid((unsigned)((p.M + rows - 1) / rows)), block(plan.tpr <= 64 ? kThreads : plan.tpr);
  const auto kernel = plan.tpr == 16   ? rmsnorm_kernel<16, 1, RES, NT>
                      : plan.tpr == 32 ? rmsnorm_kernel<32, 1, RES, NT>
                      : plan.tpr == 64 ? rmsnorm_kernel<64, 1, RES, NT>
                      : plan.vpl == 1  ? rmsnorm_kernel<0, 1, RES, NT>
                      : plan.vpl == 2  ? rmsnorm_kernel<0, 2, RES, NT>
                                       : rmsnorm_kernel<0, 4, RES, NT>;
  kernel<<<grid, block, 0, stream>>>(p);
}

}  // namespace

// One launch has at most 2^32 - 1 threads: workgroups of 256 take 4 rows at least up to
// 512 columns, those of 1024 at most one row.
bool rmsnorm_fits(int64_t M, int64_t K) {
  constexpr int64_t kLimit = ((int64_t)1 << 32) - 1;
  return K <= kMaxK && M <= (K <= 512 ? kLimit / kThreads * 4 : kLimit / kMaxThreads);
}

hipError_t launch_rmsnorm(const RmsNorm& p, hipStream_t stream) {
  const int64_t bytes = p.M * p.K * (2 + (!p.res ? 0 : p.res_f32 ? 8 : 4) + (p.y ? 2 : 0) + (p.q ? 1 : 0));
  const bool nt = bytes >= kHintBytes;
  if (p.res == nullptr) nt ? launch_fwd<0, true>(p, stream) : launch_fwd<0, false>(p, stream);
  else if (p.res_f32) nt ? launch_fwd<2, true>(p, stream) : launch_fwd<2, false>(p, stream);
  else nt ? launch_fwd<1, true>(p, stream) : launch_fwd<1, false>(p, stream);
  return hipGetLastError();
}

// ----------------------------------------------------------------------------
// gradient
//   g = dy * w, r = 1 / sqrt(mean(h^2) + eps)
//   dx = r * (g - h * r^2 * mean(g * h)) + dres,  dw = sum over rows of dy * h * r
// A workgroup goes through rows m, m + grid, ..., keeps its part of dw in
// registers and leaves it in the workspace; a second kernel adds the parts in a
// fixed order.  4096 x 7168 with dres: 235 MB and 29 MB of parts, 44 us and 5.2 for the
// parts, together 49.5 (5.3 TB/s of both).  Two rows at a time in workgroups of twice
// the size, and half the parts: 50.1; 1024 parts 56.6, 256 56.7.
// ----------------------------------------------------------------------------
namespace {

// Parts of dw at most: each costs what a row does (written and read again as float32), and fewer leave CUs idle.
// Below 1024 rows two to a part, as long as that leaves 128: 512 rows of 7168 14.9 us, in 512 parts 17.2, in 128 15.6;
// 256 rows 11.4, in 256 parts 12.4.
constexpr int kBwdGroups = 512, kBwdFew = 128;
constexpr int kBwdThreads = 512;      // of a workgroup at most: 256 registers a lane

// as plan_of, with at most kBwdThreads where a row is held
RowPlan bwd_plan_of(int64_t K) {
  const int64_t nv = K / 8;
  if (nv <= 64) return plan_of(K);
  if (nv > 4 * kBwdThreads) return {kMaxThreads, 0};         // rows read twice
  const int vpl = nv <= kBwdThreads ? 1 : nv <= 2 * kBwdThreads ? 2 : 4;
  return {(int)((nv + 64 * vpl - 1) / (64 * vpl)) * 64, vpl};
}

// rows that a workgroup takes at a time
int rows_at_once(const RowPlan& plan) { return plan.tpr <= 64 ? kThreads / plan.tpr : 1; }
int64_t bwd_groups(int64_t M, int64_t K) {
  const int rows = rows_at_once(bwd_plan_of(K));
  const int64_t units = (M + rows - 1) / rows;
  return std::min<int64_t>(std::max((units + 1) / 2, std::min<int64_t>(units, kBwdFew)), kBwdGroups);
}

}  // namespace

namespace {

// 8 elements as they lie in memory: they are held so, and made floats where they are used
template <bool F32>
struct Raw8 {
  uint4 u[F32 ? 2 : 1];
  template <bool NT>
  __device__ __forceinline__ void load(const void* p, int64_t v) {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) {
      const uint4* at = (const uint4*)p + (F32 ? 2 * v + i : v);
      u[i] = NT ? load_nt(at) : *at;
    }
  }
  __device__ __forceinline__ void floats(float* f) const { floats_of<F32>(u, f); }
};

// What a lane holds of a row
template <int VPL, bool F32>
struct RowHeld {
  Raw8<F32> h[VPL], e[VPL];
  Raw8<false> d[VPL];
  template <bool NT, bool RES>
  __device__ __forceinline__ void load(const RmsNormBwd& p, int64_t m, int j, int v) {
    h[j].template load<NT>((const char*)p.h + m * p.ld_h * (F32 ? 4 : 2), v);
    d[j].template load<NT>((const char*)p.dy + m * p.K * 2, v);
    if (RES && p.dres) e[j].template load<NT>((const char*)p.dres + m * p.K * (F32 ? 4 : 2), v);
  }
};

}  // namespace

// HELD: a lane holds VPL vectors of its row; rows too wide for that are read twice
// (the second time from L2), vector by vector, and dw lies in LDS.  (To ask for the
// next row before this one's sums are waited for costs the registers of half the
// waves: 4096 x 7168 59 us instead of 52.)
template <int TPR, int VPL, bool HELD, bool F32, bool W_F32, bool NT>
__global__ __launch_bounds__(TPR ? kThreads : HELD ? kBwdThreads : kMaxThreads) void rmsnorm_bwd_kernel(
    const RmsNormBwd p, float* parts) {
  __shared__ float red[4][kMaxThreads / 64];
  __shared__ float rows_dw[TPR ? kThreads * 8 : 1];
  __shared__ float4 wide_dw[HELD ? 1 : kMaxK / 4];
  const int tpr = TPR ? TPR : (int)blockDim.x;
  const int lane = TPR ? (int)threadIdx.x % TPR : (int)threadIdx.x;
  const int rows = TPR ? kThreads / TPR : 1;
  const int mine = TPR ? (int)threadIdx.x / TPR : 0;
  const int nv = (int)(p.K / 8);
  const float rk = (float)p.K;
  const int64_t step = (int64_t)gridDim.x * rows;
  constexpr int HV = HELD ? VPL : 1;
  Raw8<W_F32> w[HV];
  RowHeld<HV, F32> row;
  float dw[HV][8];
#pragma unroll
  for (int j = 0; j < HV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
  if (HELD) {
#pragma unroll
    for (int j = 0; j < HV; ++j) w[j].template load<false>(p.w, min(lane + j * tpr, nv - 1));
  } else {
    for (int v = lane; v < nv; v += tpr) wide_dw[2 * v] = wide_dw[2 * v + 1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  int turn = 0;
  for (int64_t m0 = (int64_t)blockIdx.x * rows; m0 < p.M; m0 += step, turn ^= 1) {
    const int64_t m = m0 + mine;
    float hh = 0.0f, gh = 0.0f;
    const auto add_up = [&](int j, bool on) {
      float h[8], d[8], g[8];
      row.h[j].floats(h);
      row.d[j].floats(d);
      w[j].floats(g);
      float a = 0.0f, b = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a = __builtin_fmaf(h[i], h[i], a);
        b = __builtin_fmaf(d[i] * g[i], h[i], b);
      }
      hh += on ? a : 0.0f;
      gh += on ? b : 0.0f;
    };
    if (HELD) {
#pragma unroll
      for (int j = 0; j < HV; ++j) row.template load<NT, true>(p, min(m, p.M - 1), j, min(lane + j * tpr, nv - 1));
#pragma unroll
      for (int j = 0; j < HV; ++j) add_up(j, lane + j * tpr < nv);
    } else {
#pragma unroll 2
      for (int v = lane; v < nv; v += tpr) {
        row.template load<false, false>(p, m, 0, v);
        w[0].template load<false>(p.w, v);
        add_up(0, true);
      }
    }
    // two buffers in turn: a wave may be at the next row's sums while another still reads this one's
    if (TPR) {
      hh = row_sum<TPR>(hh, nullptr);
      gh = row_sum<TPR>(gh, nullptr);
    } else {
      hh = wave_sum(hh);
      gh = wave_sum(gh);
      if ((threadIdx.x & 63) == 0) {
        red[2 * turn][threadIdx.x >> 6] = hh;
        red[2 * turn + 1][threadIdx.x >> 6] = gh;
      }
      __syncthreads();
      hh = gh = 0.0f;
      for (int i = 0; i < (int)blockDim.x / 64; ++i) {
        hh += red[2 * turn][i];
        gh += red[2 * turn + 1][i];
      }
    }
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(hh, rk) + p.eps));
    const float c = r * r * __fdiv_rn(gh, rk);
    const auto finish = [&](int j, int v, float* sum) {
      float h[8], d[8], g[8], e[8];
      row.h[j].floats(h);
      row.d[j].floats(d);
      w[j].floats(g);
      if (p.dres) row.e[j].floats(e);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float o = r * __builtin_fmaf(-h[i], c, d[i] * g[i]);
        if (p.dres) o += e[i];
        sum[i] = __builtin_fmaf(d[i], h[i] * r, sum[i]);
        e[i] = o;
      }
      store8<F32>(p.dx, m * nv + v, e);
    };
    if (HELD) {
      if (m < p.M) {
#pragma unroll
        for (int j = 0; j < HV; ++j) {
          const int v = lane + j * tpr;
          if (v >= nv) break;
          finish(j, v, dw[j]);
        }
      }
    } else {
      for (int v = lane; v < nv; v += tpr) {
        row.template load<NT, true>(p, m, 0, v);
        w[0].template load<false>(p.w, v);
        float sum[8];
        load8<true, false>(wide_dw, v, sum);
        finish(0, v, sum);
        wide_dw[2 * v] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        wide_dw[2 * v + 1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
      }
    }
  }
  if (!parts) return;
  float* out = parts + (int64_t)blockIdx.x * p.K;
  if (TPR) {
    // the rows' parts of a column lie tpr * 8 floats apart
#pragma unroll
    for (int i = 0; i < 8; ++i) rows_dw[threadIdx.x * 8 + i] = dw[0][i];
    __syncthreads();
    for (int k = threadIdx.x; k < p.K; k += kThreads) {
      float a = 0.0f;
      for (int r = 0; r < rows; ++r) a += rows_dw[r * tpr * 8 + k];
      out[k] = a;
    }
  } else if (HELD) {
#pragma unroll
    for (int j = 0; j < HV; ++j) {
      const int v = lane + j * tpr;
      if (v >= nv) break;
      ((float4*)out)[2 * v] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
      ((float4*)out)[2 * v + 1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
    }
  } else {
    for (int v = lane; v < nv; v += tpr)
      for (int i = 0; i < 2; ++i) ((float4*)out)[2 * v + i] = wide_dw[2 * v + i];
  }
}

// dw[k] = the sum of G parts: of 32 columns (a line of each part), 32 groups of 8 threads take every 32nd part, 8
// loads at a time; then their sums in order.
constexpr int kDwGroups = 32;
__global__ __launch_bounds__(256) void rmsnorm_dw_kernel(const float* __restrict__ parts, float* __restrict__ dw,
                                                          int64_t G, int64_t K) {
  __shared__ float4 sums[kDwGroups][8];
  const int col = threadIdx.x & 7, grp = threadIdx.x >> 3;
  const int64_t c4 = (int64_t)blockIdx.x * 8 + col;          // K is a multiple of 32
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float4* p = (const float4*)parts + c4;
  for (int64_t g0 = grp; g0 < G; g0 += 8 * kDwGroups) {
    float4 b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = p[min(g0 + i * kDwGroups, G - 1) * (K / 4)];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (g0 + i * kDwGroups < G) a.x += b[i].x, a.y += b[i].y, a.z += b[i].z, a.w += b[i].w;
  }
  sums[grp][col] = a;
  __syncthreads();
  if (grp == 0) {
    for (int g = 1; g < kDwGroups; ++g) {
      const float4 b = sums[g][col];
      a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
    }
    ((float4*)dw)[c4] = a;
  }
}

int64_t rmsnorm_bwd_workspace_bytes(int64_t M, int64_t K) {
  const int64_t G = bwd_groups(M, K);
  return G > 1 ? G * K * 4 : 0;                              // one workgroup writes dw itself
}

template <bool F32, bool W_F32, bool NT>
static void launch_bwd_of(const RmsNormBwd& p, float* parts, hipStream_t stream) {
  const RowPlan plan = bwd_plan_of(p.K);
  const dim3 grid((unsigned)bwd_groups(p.M, p.K)), block(plan.tpr <= 64 ? kThreads : plan.tpr);
  const auto kernel = plan.tpr == 16  ? rmsnorm_bwd_kernel<16, 1, true, F32, W_F32, NT>
                      : plan.tpr == 32 ? rmsnorm_bwd_kernel<32, 1, true, F32, W_F32, NT>
                      : plan.tpr == 64 ? rmsnorm_bwd_kernel<64, 1, true, F32, W_F32, NT>
                      : plan.vpl == 1  ? rmsnorm_bwd_kernel<0, 1, true, F32, W_F32, NT>
                      : plan.vpl == 2  ? rmsnorm_bwd_kernel<0, 2, true, F32, W_F32, NT>
                      : plan.vpl == 4  ? rmsnorm_bwd_kernel<0, 4, true, F32, W_F32, NT>
                                       : rmsnorm_bwd_kernel<0, 0, false, F32, W_F32, NT>;
  kernel<<<grid, block, 0, stream>>>(p, parts);
}

template <bool F32, bool W_F32>
static void launch_bwd(const RmsNormBwd& p, float* parts, hipStream_t stream) {
  const int64_t size = F32 ? 4 : 2, bytes = p.M * p.K * (2 + (p.dres ? 3 : 2) * size);
  if (bytes >= kHintBytes) launch_bwd_of<F32, W_F32, true>(p, parts, stream);
  else launch_bwd_of<F32, W_F32, false>(p, parts, stream);
}

hipError_t launch_rmsnorm_bwd(const RmsNormBwd& p, hipStream_t stream) {
  const int64_t G = bwd_groups(p.M, p.K);
  float* parts = !p.dw ? nullptr : G > 1 ? (float*)p.workspace : p.dw;
  if (G > 0) {
    if (p.h_f32) p.w_f32 ? launch_bwd<true, true>(p, parts, stream) : launch_bwd<true, false>(p, parts, stream);
    else p.w_f32 ? launch_bwd<false, true>(p, parts, stream) : launch_bwd<false, false>(p, parts, stream);
  }
  if (p.dw && G != 1)                                        // no rows: dw is zero
    rmsnorm_dw_kernel<<<dim3((unsigned)(p.K / 32)), dim3(256), 0, stream>>>((const float*)p.workspace, p.dw, G, p.K);
  return hipGetLastError();
}

}  // namespace fp8bs
