// mla_attention.hip -- attention of new tokens over a paged MLA latent cache
// for gfx950: step 6 of the absorb attention ("DeepSeek-V3 Administrator &
// Developer Guide" 8.3), between the two products of mla.hip.
//
// All heads of a token share one key per cached token, the normalised latent
// c_j (R = 512) beside the rotated part k_j (64), and the latent is the value
// too:
//   s[r, j] = scale * (q_lat[r] . c_j + q_rope[r] . k_j),   j < end(r)
//   out[r]  = sum_j softmax_j(s[r, :]) c_j
// with a row r = (token, head).  The rows of a sequence, token-major, are cut
// into tiles of M rows whose cached tokens are streamed once per tile.
//
// Softmax in one pass, in base 2: a running maximum m, sum l and the
// accumulator O.  O and l are rescaled only when a tile's maximum exceeds m
// by more than kLazy = 8: until then probabilities are taken against the older
// m and reach at most 2^8, which costs no precision (bf16 and float32 round
// relatively) and leaves the accumulators alone.
//
// MFMA: v_mfma_f32_16x16x32_bf16, D[16 x 16] = X[16 x 32] . Y[32 x 16]; lane
// (g = l / 16, n = l % 16) supplies row n of X and column n of Y at K values
// 8g .. 8g+7, and register r of its result is D[4g + r][n].
//   scores   X = 16 cached tokens, Y = 16 query rows: a lane holds tokens
//            4g + r of one query row, so a row's maximum and sum are in-lane
//            but for the four g.
//   output   X = 16 latent channels (transposed reads), Y = the probabilities:
//            over two score tiles (tokens 0..15 and 16..31) a lane owns tokens
//            4g + r and 16 + 4g + r, which are taken as its K values 8g + r
//            and 8g + 4 + r, so probabilities go from the score's registers to
//            the operand without crossing lanes.  The latents are read in the
//            same order by two 4-token transposed LDS reads.
//
// A wave carries 16 RT query rows (Q in registers) over 32 cached tokens at a
// time; RW waves take different rows of the same tokens and TW waves different
// tokens of the same rows.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "device_common.h"
#include "launch.h"

namespace fp8bs {

namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) v4u lds_v4u;

constexpr int kR = 512;                 // latent width
constexpr int kD = 64;                  // rotated width
constexpr int kTok = 32;                // cached tokens per wave and step
constexpr int kSteps = (kR + kD) / 32;  // K steps of a score: 16 latent, 2 rotated
constexpr int kCt = kR / 16;            // channel tiles of the output
constexpr int kRowB = kR * 2;           // bytes of a latent row in LDS
constexpr int kRopeB = kD * 2;
constexpr int kLatB = kTok * kRowB;
constexpr int kTileB = kLatB + kTok * kRopeB;   // 36,864 bytes
constexpr float kLazy = 8.0f;
constexpr float kNegInf = -__builtin_huge_valf();

struct AttnParams {
  const uint16_t* q_lat;
  const uint16_t* q_rope;
  const uint8_t* latent;    // bf16 or e4m3 [P, ps, 512]
  const float* lat_scale;   // e4m3: [P, ps, 4]
  const uint16_t* rope;     // bf16 [P, ps, 64]
  const int32_t* table;     // [B, W]
  const int32_t* cu_q;      // [B + 1]
  const int32_t* lens;      // [B]
  void* out;                // [T, H, 512]
  float* lse;               // [T, H] or null
  int64_t ldq_t, ldq_h, ldr_t, ldr_h;
  float scale2;             // scale * log2(e)
  int T, H, B, W, P, ps;
  int causal, out_f32;
};

// The 16-byte chunk c of latent row t sits at slot c ^ lat_swz(t), and of
// rope row t at c ^ rope_swz(t).  A linear map of the token's bits chosen for
// the LDS's rule (a b128 read is served in four cycles of the 16 lanes of a
// half-wave with equal parity of lane bits 2..4, a b64 read by half-waves, over
// 64 banks): the score reads (16 tokens x chunks g of a K step) and the
// transposed reads (8 tokens x 2 chunks) both touch 16 distinct slots a cycle.
__device__ __forceinline__ int lat_swz(int t) { return ((t & 7) << 1) ^ ((t & 8) ? 9 : 0); }
__device__ __forceinline__ int rope_swz(int t) { return ((t & 2) << 1) | ((t & 4) >> 1) | ((t & 4) >> 2); }

__device__ __forceinline__ v4f mfma_bf16(v8bf x, v8bf y, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t lds_at(const void* q) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)q;
}
__device__ __forceinline__ v8bf lds_b128(uint32_t at, int off) {
  return __builtin_bit_cast(v8bf, *((const lds_v4u*)(uintptr_t)at + off / 16));
}
// 4 tokens x 16 channels, transposed, twice: tokens 4g .. + 3 and 16 + 4g .. + 3
__device__ __forceinline__ v8bf lds_tr(uint32_t at, int off) {
  typedef short v8s __attribute__((ext_vector_type(8)));
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)at + off / 8);
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)at + (off + 16 * kRowB) / 8);
  return __builtin_bit_cast(v8bf, (v8s)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The output accumulators: tile (rt, ct) of a wave is the AGPRs 4 i .. 4 i + 3
// with i = kCt rt + ct, 256 of them per lane with RT = 2, named in the
// instructions below.  Left to the compiler they would be VGPRs (the rare
// rescale is VALU work, which cannot take AGPRs), and with Q's 144 registers
// that spilled 230 of them to memory.  The source is built so that the
// compiler itself puts nothing into AGPRs (its own MFMAs in the VGPR form, and
// less than 256 VGPRs live), which a test of the listing checks.
// Wait states: a VALU result may be an MFMA operand two cycles later (s_nop 1);
// an MFMA's result may be read by another kind of instruction 19 cycles later.
template <int I>
__device__ __forceinline__ void acc_mfma(v8bf x, v8bf y) {
  asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 a[%0:%1], %2, %3, a[%0:%1]"
               :: "n"(4 * I), "n"(4 * I + 3), "v"(x), "v"(y));
}
__device__ __forceinline__ void acc_settle() { asm volatile("s_nop 15\n\ts_nop 7"); }
template <int I>
__device__ __forceinline__ v4f acc_read() {
  float a, b, c, d;
  asm volatile("v_accvgpr_read_b32 %0, a[%4]\n\tv_accvgpr_read_b32 %1, a[%5]\n\t"
               "v_accvgpr_read_b32 %2, a[%6]\n\tv_accvgpr_read_b32 %3, a[%7]"
               : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d) : "n"(4 * I), "n"(4 * I + 1), "n"(4 * I + 2), "n"(4 * I + 3));
  return v4f{a, b, c, d};
}
template <int I>
__device__ __forceinline__ void acc_write(v4f v) {
  asm volatile("v_accvgpr_write_b32 a[%4], %0\n\tv_accvgpr_write_b32 a[%5], %1\n\t"
               "v_accvgpr_write_b32 a[%6], %2\n\tv_accvgpr_write_b32 a[%7], %3"
               :: "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "n"(4 * I), "n"(4 * I + 1), "n"(4 * I + 2), "n"(4 * I + 3));
}
// calls f with the constants 0 .. N-1
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unroll(const F& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unroll<N, I + 1>(f);
  }
}
// tells the compiler how many registers a kernel of RT row tiles takes
template <int RT>
__device__ __forceinline__ void acc_reserve() {
  if constexpr (RT == 1) asm volatile("" ::: "a127");
  else asm volatile("" ::: "a255");
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// a sequence of the batch; every field is clamped to what the buffers hold
struct Seq {
  int q0, nq, len;
};
__device__ __forceinline__ Seq load_seq(const AttnParams& p, int b) {
  Seq s;
  s.q0 = clampi(p.cu_q[b], 0, p.T);
  s.nq = clampi(p.cu_q[b + 1], s.q0, p.T) - s.q0;
  s.len = (int)min((int64_t)max(p.lens[b], 0), (int64_t)p.W * p.ps);
  return s;
}

// cached tokens that query token i of a sequence sees
__device__ __forceinline__ int visible(const AttnParams& p, const Seq& s, int i) {
  return p.causal ? clampi(s.len - s.nq + i + 1, 0, s.len) : s.len;
}

template <int RT, int RW, int TW, bool FP8>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
mla_attention_kernel(AttnParams p) {
  constexpr int M = 16 * RT * RW;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[std::max(kTileB * TW, TW > 1 ? 4 * 16 * kR * 4 : 0)];
  const int lane = threadIdx.x & 63;
  const int n = lane & 15, g = lane >> 4;
  const int wave = threadIdx.x >> 6;
  const int rw = wave % RW, tw = wave / RW;
  uint8_t* const tile = smem + tw * kTileB;

  // this workgroup's row tile
  int b = 0, rt0 = blockIdx.x;
  Seq sq;
  for (;; ++b) {
    if (b >= p.B) return;
    sq = load_seq(p, b);
    const int64_t nrt = ((int64_t)sq.nq * p.H + M - 1) / M;
    if (rt0 < nrt) break;
    rt0 -= (int)nrt;
  }
  const int rows = sq.nq * p.H;
  const int r_tile = rt0 * M;
  const int r_last = min(r_tile + M, rows) - 1;
  const int end_max = visible(p, sq, r_last / p.H);
  const int end_min = visible(p, sq, r_tile / p.H);

  // query rows of this wave: their operands, and the tokens they see
  v8bf q[RT][kSteps];
  int end[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = min(r_tile + (rw * RT + rt) * 16 + n, r_last);
    const int i = r / p.H, h = r - i * p.H;
    end[rt] = visible(p, sq, i);
    const uint16_t* ql = p.q_lat + (sq.q0 + i) * p.ldq_t + h * p.ldq_h + 8 * g;
    const uint16_t* qr = p.q_rope + (sq.q0 + i) * p.ldr_t + h * p.ldr_h + 8 * g;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      q[rt][s] = __builtin_bit_cast(v8bf, *reinterpret_cast<const v4u*>(s < kR / 32 ? ql + 32 * s : qr + 32 * s - kR));
  }

  float m[RT], l[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = kNegInf;
    l[rt] = 0.0f;
  }
  acc_reserve<RT>();
  unroll<RT * kCt>([&](auto i) { acc_write<i>(v4f{0.0f, 0.0f, 0.0f, 0.0f}); });

  // The operand reads' LDS addresses.  A latent chunk's swizzle touches the low
  // four bits of its index alone, so K steps k, k + 4, .. and channel tiles
  // ct, ct + 8, .. share a base, and both halves of the 32 tokens do.
  const uint32_t tile_at = lds_at(tile);
  uint32_t kat[4], kro[2], vat[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) kat[k] = tile_at + n * kRowB + (((4 * k + g) ^ lat_swz(n)) << 4);
#pragma unroll
  for (int k = 0; k < 2; ++k) kro[k] = tile_at + kLatB + n * kRopeB + (((4 * k + g) ^ rope_swz(n)) << 4);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int t = 4 * g + (n >> 2);                  // the lane points at this token, 4 channels from 4 (n % 4)
    vat[k] = tile_at + t * kRowB + (((2 * k + ((n & 3) >> 1)) ^ lat_swz(t)) << 4) + ((n & 1) << 3);
  }

  const int32_t* trow = p.table + (int64_t)b * p.W;
  for (int t0 = 0; t0 < end_max; t0 += kTok * TW) {
    const int tb = t0 + tw * kTok;                   // first token of this wave
    __syncthreads();
    // Lane j < 32 finds token tb + j; tokens past the last visible one load that one again,
    // so masked places hold finite values and nothing behind the sequence is read.
    const int tok = min(tb + (lane & 31), end_max - 1);
    const int pg = clampi(trow[(uint32_t)tok / (uint32_t)p.ps], 0, p.P - 1);
    const int64_t row = (int64_t)pg * p.ps + (uint32_t)tok % (uint32_t)p.ps;
    const int row_lo = (int)row;                     // P * ps < 2^31
    if (FP8) {
#pragma unroll 4
      for (int i = 0; i < kTok / 2 / RW; ++i) {
        const int t = 2 * (i * RW + rw) + (lane >> 5), c = lane & 31;
        const int64_t src = __shfl(row_lo, t);
        const v4u w = *reinterpret_cast<const v4u*>(p.latent + src * kR + 16 * c);
        const float sc = p.lat_scale[src * (kR / 128) + (c >> 3)];
        uint8_t* dst = tile + t * kRowB;
        *reinterpret_cast<v4u*>(dst + (((2 * c) ^ lat_swz(t)) << 4)) = __builtin_bit_cast(v4u, dequant8_bf16(w.x, w.y, sc));
        *reinterpret_cast<v4u*>(dst + (((2 * c + 1) ^ lat_swz(t)) << 4)) = __builtin_bit_cast(v4u, dequant8_bf16(w.z, w.w, sc));
      }
    } else {
#pragma unroll 8
      for (int i = 0; i < kTok / RW; ++i) {
        const int t = i * RW + rw;
        const int64_t src = __shfl(row_lo, t);
        const v4u w = *reinterpret_cast<const v4u*>(p.latent + src * kRowB + 16 * lane);
        *reinterpret_cast<v4u*>(tile + t * kRowB + ((lane ^ lat_swz(t)) << 4)) = w;
      }
    }
#pragma unroll
    for (int i = 0; i < kTok / 8 / RW; ++i) {
      const int t = 8 * (i * RW + rw) + (lane >> 3), c = lane & 7;
      const int64_t src = __shfl(row_lo, t);
      const v4u w = *reinterpret_cast<const v4u*>(reinterpret_cast<const uint8_t*>(p.rope) + src * kRopeB + 16 * c);
      *reinterpret_cast<v4u*>(tile + kLatB + t * kRopeB + ((c ^ rope_swz(t)) << 4)) = w;
    }
    __syncthreads();

    // scores of 32 tokens
    v4f s[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const v8bf x = k < kR / 32 ? lds_b128(kat[k & 3], (k >> 2) * 256 + tt * 16 * kRowB)
                                   : lds_b128(kro[k & 1], tt * 16 * kRopeB);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) s[rt][tt] = mfma_bf16(x, q[rt][k], s[rt][tt]);
      }

    // probabilities
    v8bf pr[RT];
    unroll<RT>([&](auto rt) {
      float x[8];
      float top = kNegInf;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = s[rt][e >> 2][e & 3] * p.scale2;
        if (tb + kTok > end_min && tb + 16 * (e >> 2) + 4 * g + (e & 3) >= end[rt]) x[e] = kNegInf;
        top = fmaxf(top, x[e]);
      }
      if (__any(top > m[rt] + kLazy)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float mn = fmaxf(m[rt], top);
        const float a = mn == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - mn);
        m[rt] = mn;
        l[rt] *= a;
        acc_settle();
        unroll<kCt>([&](auto ct) { acc_write<kCt * rt + ct>(acc_read<kCt * rt + ct>() * a); });
      }
      const float base = m[rt] == kNegInf ? 0.0f : m[rt];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = __builtin_amdgcn_exp2f(x[e] - base);
        l[rt] += x[e];
      }
      const v4u u = {pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]), pack2_bf16(x[4], x[5]), pack2_bf16(x[6], x[7])};
      pr[rt] = __builtin_bit_cast(v8bf, u);
    });

    // output
    unroll<kCt>([&](auto ct) {
      const v8bf x = lds_tr(vat[ct & 7], (ct >> 3) * 256);
      unroll<RT>([&](auto rt) { acc_mfma<kCt * rt + ct>(x, pr[rt]); });
    });
  }
  acc_settle();

  // the row's sum over the four g, then over the token waves
  float* const red = reinterpret_cast<float*>(smem);   // [4 waves][m 16, l 16], then [4 waves][512][16 rows]
  unroll<RT>([&](auto rt) {
    l[rt] += __shfl_xor(l[rt], 16);
    l[rt] += __shfl_xor(l[rt], 32);
    float w = 1.0f;
    float mt = m[rt], lt = l[rt];
    if constexpr (TW > 1) {
      __syncthreads();
      if (g == 0) {
        red[wave * 32 + n] = m[rt];
        red[wave * 32 + 16 + n] = l[rt];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < TW; ++k) mt = fmaxf(mt, red[(k * RW + rw) * 32 + n]);
      lt = 0.0f;
#pragma unroll
      for (int k = 0; k < TW; ++k) {
        const float mk = red[(k * RW + rw) * 32 + n];
        if (mk > kNegInf) lt += red[(k * RW + rw) * 32 + 16 + n] * __builtin_amdgcn_exp2f(mk - mt);
      }
      w = m[rt] > kNegInf ? __builtin_amdgcn_exp2f(m[rt] - mt) : 0.0f;
      __syncthreads();
      float* ow = red + wave * 16 * kR;
      unroll<kCt>([&](auto ct) {
        const v4f v = acc_read<kCt * rt + ct>() * w;
#pragma unroll
        for (int e = 0; e < 4; ++e) ow[(16 * ct + 4 * g + e) * 16 + n] = v[e];
      });
      __syncthreads();
    }
    // token wave tw adds and stores the channel tiles tw kCt / TW ..
    const int r = r_tile + (rw * RT + rt) * 16 + n;
    if (r <= r_last) {
      const float inv = lt > 0.0f ? 1.0f / lt : 0.0f;
      const int64_t orow = (int64_t)sq.q0 * p.H + r;
      if (tw == 0 && g == 0 && p.lse)
        p.lse[orow] = lt > 0.0f ? (mt + __builtin_log2f(lt)) * 0.693147180559945309f : kNegInf;
      unroll<kCt / TW>([&](auto i) {
        const int ct = tw * (kCt / TW) + i;
        v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (TW > 1) {
#pragma unroll
          for (int k = 0; k < TW; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += red[(k * RW + rw) * 16 * kR + (16 * ct + 4 * g + e) * 16 + n];
        } else {
          v = acc_read<kCt * rt + i>();
        }
        v *= inv;
        const int64_t at = orow * kR + 16 * ct + 4 * g;
        if (p.out_f32) *reinterpret_cast<v4f*>(static_cast<float*>(p.out) + at) = v;
        else *reinterpret_cast<v2u*>(static_cast<uint16_t*>(p.out) + at) = v2u{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])};
      });
    }
  });
}

}  // namespace

int64_t mla_attention_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_mla_attention(const MlaAttention& a, hipStream_t stream) {
  AttnParams p{};
  p.q_lat = static_cast<const uint16_t*>(a.q_lat);
  p.q_rope = static_cast<const uint16_t*>(a.q_rope);
  p.latent = static_cast<const uint8_t*>(a.latent);
  p.lat_scale = a.lat_scale;
  p.rope = static_cast<const uint16_t*>(a.rope);
  p.table = a.table;
  p.cu_q = a.cu_q;
  p.lens = a.lens;
  p.out = a.out;
  p.lse = a.lse;
  p.ldq_t = a.ldq_t;
  p.ldq_h = a.ldq_h;
  p.ldr_t = a.ldr_t;
  p.ldr_h = a.ldr_h;
  p.scale2 = a.scale * 1.4426950408889634f;
  p.T = (int)a.T;
  p.H = (int)a.H;
  p.B = (int)a.B;
  p.W = (int)a.W;
  p.P = (int)a.P;
  p.ps = (int)a.ps;
  p.causal = a.causal;
  p.out_f32 = a.out_f32;
  // rows of an average sequence decide the tile
  const int64_t rows = a.T * a.H, per = rows / a.B;
#define FP8BS_ATTN(RT_, RW_, TW_, F8_)                                                          \
  {                                                                                             \
    constexpr int M_ = 16 * RT_ * RW_;                                                          \
    const dim3 grid((unsigned)((rows + M_ - 1) / M_ + a.B));                                    \
    hipLaunchKernelGGL((mla_attention_kernel<RT_, RW_, TW_, F8_>), grid, dim3(256), 0, stream, p); \
  }
#define FP8BS_ATTN_F(RT_, RW_, TW_)            \
  {                                            \
    if (a.fp8) FP8BS_ATTN(RT_, RW_, TW_, true) \
    else FP8BS_ATTN(RT_, RW_, TW_, false)      \
  }
  if (per >= 96) FP8BS_ATTN_F(2, 4, 1)
  else if (per >= 48) FP8BS_ATTN_F(2, 2, 2)
  else if (per >= 24) FP8BS_ATTN_F(2, 1, 4)
  else FP8BS_ATTN_F(1, 1, 4)
#undef FP8BS_ATTN_F
#undef FP8BS_ATTN
  return hipGetLastError();
}

}  // namespace fp8bs
