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
constexpr int kCodeB = kTok * kR;                // the same 32 tokens of an FP8 cache as they come:
constexpr int kRawB = kCodeB + kTok * kRopeB + 1024;   // codes, rope, scales (512 bytes, written twice)
constexpr int kAhead = 6;
constexpr float kLazy = 8.0f;
constexpr float kLn2 = 0.693147180559945309f;
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
  uint32_t ps_mul;          // tok / ps = tok * ps_mul >> ps_shift for tok < 2^31
  int ps_shift;
  // workspace: [grid] Meta, then [grid][2][M] lse (base 2), then [grid][2][M][512] normalised output parts
  struct Meta* meta;
  float* part_lse;
  float* part_out;
  int T, H, B, W, P, ps;
  int causal, out_f32;
};

// what a workgroup leaves for the join: the row tile that it begins and does not finish
struct Meta {
  int64_t row;      // its first row of [T * H]
  int rows, parts;  // parts = 0: none.  Part 0 is this workgroup's, part k the k-th next one's.
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

// four consecutive output values
__device__ __forceinline__ void store4(const AttnParams& p, int64_t at, v4f v) {
  if (p.out_f32) *reinterpret_cast<v4f*>(static_cast<float*>(p.out) + at) = v;
  else *reinterpret_cast<v2u*>(static_cast<uint16_t*>(p.out) + at) = v2u{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])};
}

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

// Direct global -> LDS loads, 16 bytes a lane: lane i's bytes land at lds + 16 i.
// In assembly, so that the compiler does not make every LDS read wait for all
// of them; completion is awaited with wait_vmcnt.
__device__ __forceinline__ void dma_row(const void* base, uint32_t off, uint32_t lds) {
  // five wait states, should a VALU instruction have written the base's scalar registers just before
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void dma_lanes(const void* at, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(at) : "memory", "m0");
}
template <int n>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8));
  asm volatile("" ::: "memory");
}
// workgroup barrier that orders LDS accesses only
__device__ __forceinline__ void barrier_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// exclusive prefix sum over the workgroup's 256 threads; total gets the sum
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sums, int64_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) sums[wave] = x;
  __syncthreads();
  int64_t base = 0;
  total = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k < wave) base += sums[k];
    total += sums[k];
  }
  return base + x - v;
}

// ---------------------------------------------------------------------------
// The work split.  The grid is one workgroup per CU, whatever the batch.  The
// row tiles of all sequences, in order, cost kStart + (steps of 32 TW cached
// tokens) each; the sum of the costs is cut into equal shares, and workgroup w
// works through share w: the end of one tile's tokens, whole tiles, the
// beginning of another's.  So long and short sequences, few rows and many, all
// fill the card evenly, from lengths that only the device knows.  A tile that
// several workgroups share is joined by join_kernel from at most two parts per
// workgroup.  Every workgroup computes the split itself: two prefix sums, over
// the sequences (row tiles) and over the row tiles (costs).
// ---------------------------------------------------------------------------
constexpr int kStart = 2;    // a tile's queries and output, in steps
constexpr int kLeast = 4;    // a share is no smaller, so that short work is not cut to pieces
// A cut this near a tile's edge moves to it: a split costs the writing and
// reading of M rows of float32 twice, about M / 16 steps' time.
template <int M>
__device__ __forceinline__ int slack(int64_t total, int shares) { return (int)min((int64_t)(M / 16), total / shares / 4); }

struct Cut {          // a place between two steps
  int tile;           // row tile of the batch
  int b, in_seq;      // its sequence, its index there
  int step;
  int64_t end;        // costs up to the tile's end
};

// values that all lanes share, moved to scalar registers
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}
__device__ __forceinline__ Cut uniform(const Cut& c) {
  return Cut{uniform(c.tile), uniform(c.b), uniform(c.in_seq), uniform(c.step), uniform(c.end)};
}

template <int M, int STEP>
struct Plan {
  Cut lo, hi;
  int64_t total;
  int shares, near;

  static __device__ int tile_cost(const AttnParams& p, const Seq& s, int in_seq) {
    const int r = (int)min((int64_t)(in_seq + 1) * M, (int64_t)s.nq * p.H) - 1;
    return kStart + (visible(p, s, r / p.H) + STEP - 1) / STEP;
  }

  // false: this workgroup has no share
  __device__ bool make(const AttnParams& p, int w, uint8_t* smem) {
    int64_t* sums = reinterpret_cast<int64_t*>(smem);
    Cut* cut = reinterpret_cast<Cut*>(smem + 64);
    int* first = reinterpret_cast<int*>(smem + 256);       // [B + 1] row tiles before each sequence
    const int tid = threadIdx.x;
    const int per_b = (p.B + 255) / 256;
    const int b0 = min(tid * per_b, p.B), b1 = min(b0 + per_b, p.B);
    int64_t mine = 0, sum;
    for (int b = b0; b < b1; ++b) mine += ((int64_t)load_seq(p, b).nq * p.H + M - 1) / M;
    int64_t at = block_scan(mine, sums, sum);
    const int tiles = (int)sum;
    for (int b = b0; b < b1; ++b) {
      first[b] = (int)at;
      at += ((int64_t)load_seq(p, b).nq * p.H + M - 1) / M;
    }
    if (tid == 0) first[p.B] = tiles;
    __syncthreads();

    const int per_t = (tiles + 255) / 256;
    const int t0 = min(tid * per_t, tiles), t1 = min(t0 + per_t, tiles);
    int b = 0;
    for (int n = p.B; n > 1;) {                            // the last b with first[b] <= t0
      const int half = n / 2;
      if (first[b + half] <= t0) b += half;
      n -= half;
    }
    mine = 0;
    const int bs = b;
    Seq s = load_seq(p, b);
    for (int t = t0; t < t1; ++t) {
      while (t >= first[b + 1]) s = load_seq(p, ++b);
      mine += tile_cost(p, s, t - first[b]);
    }
    int64_t base = block_scan(mine, sums, total);
    shares = (int)max((int64_t)1, min((int64_t)gridDim.x, total / kLeast));
    if (w >= shares || total == 0) return false;

    near = uniform(slack<M>(total, shares));
    const int64_t want[2] = {total * w / shares, total * (w + 1) / shares};
    if (t1 == tiles && t0 < t1 && want[1] == total) cut[1] = Cut{tiles, p.B, 0, 0, total};
    if (t0 < t1 && ((want[0] >= base && want[0] < base + mine) || (want[1] >= base && want[1] < base + mine))) {
      b = bs;
      s = load_seq(p, b);
      for (int t = t0; t < t1; ++t) {
        while (t >= first[b + 1]) s = load_seq(p, ++b);
        const int c = tile_cost(p, s, t - first[b]);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (want[k] >= base && want[k] < base + c) {
            const int at = (int)(want[k] - base);
            // (tile t + 1 may be the next sequence's first: the share that begins there looks)
            if (at <= kStart + near) cut[k] = Cut{t, b, t - first[b], 0, base + c};
            else if (at >= c - near) cut[k] = Cut{t + 1, b, t + 1 - first[b], 0, base + c};
            else cut[k] = Cut{t, b, t - first[b], at - kStart, base + c};
          }
        base += c;
      }
    }
    __syncthreads();
    lo = uniform(cut[0]);
    hi = uniform(cut[1]);
    total = uniform(total);
    shares = uniform(shares);
    __syncthreads();
    return true;
  }
};

// the next sequence after b that has new tokens (there is one)
__device__ __forceinline__ int next_seq(const AttnParams& p, int b) {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  for (++b; b < p.B; b += 64) {
    const uint64_t some = __ballot(b + lane < p.B && load_seq(p, min(b + lane, p.B - 1)).nq > 0);
    if (some) return b + __ffsll((unsigned long long)some) - 1;
  }
  return p.B - 1;
}

// Stages of cached tokens under way per token wave, and LDS: with one stage (RW
// = 1) every wave loads, waits and computes by itself, no barrier, the waves
// covering each other's waits; else a ring of ST stages.  An FP8 cache's codes
// come in as they are and are spread to bf16 in LDS once for all row waves;
// with RW = 1 they wait in registers.
template <int RW, int TW, bool FP8>
constexpr int stages() { return RW == 1 ? 1 : TW == 1 ? 4 : 2; }
template <int RW, int TW, bool FP8>
constexpr int lds_bytes() {
  constexpr int st = stages<RW, TW, FP8>();
  constexpr int n = FP8 ? TW * (kTileB + (RW == 1 ? 0 : st * kRawB)) : TW * st * kTileB;
  return TW > 1 ? std::max(n, 4 * 16 * kR * 4) : n;   // the token waves' accumulators meet here
}

template <int RT, int RW, int TW, bool FP8>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
mla_attention_kernel(AttnParams p) {
  constexpr int M = 16 * RT * RW, STEP = kTok * TW;
  constexpr int ST = stages<RW, TW, FP8>();
  static_assert(RW * TW == 4 && lds_bytes<RW, TW, FP8>() <= 160 * 1024, "layout");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[lds_bytes<RW, TW, FP8>()];
  const int lane = threadIdx.x & 63;
  const int n = lane & 15, g = lane >> 4;
  const int wave = uniform((int)threadIdx.x >> 6);
  const int rw = wave % RW, tw = wave / RW;
  uint8_t* const tile = smem + tw * (FP8 ? 1 : ST) * kTileB;               // bf16 tiles of this token wave
  uint8_t* const raw = smem + TW * kTileB + tw * ST * kRawB;               // FP8: its stages

  // neighbouring shares on one XCD (workgroups go round the eight): they often stream the same tokens
  const int w = gridDim.x % 8 == 0 ? (blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8 : blockIdx.x;
  if (threadIdx.x == 0) p.meta[w].parts = 0;
  Plan<M, STEP> plan;
  if (!plan.make(p, w, smem)) return;

  // The operand reads' LDS addresses.  A latent chunk's swizzle touches the low
  // four bits of its index alone and by exclusive or, so the address of K step k
  // is that of step 0 with 64 (k % 4) xored in and 256 (k / 4) added, that of
  // channel tile ct has 32 (ct % 8) xored in and 256 (ct / 8) added, and the second
  // 16 tokens are 16 rows on.
  const uint32_t tile_at = lds_at(tile);
  const uint32_t key_at = tile_at + n * kRowB + ((g ^ lat_swz(n)) << 4);
  const uint32_t key_rope_at = tile_at + kLatB + n * kRopeB + ((g ^ rope_swz(n)) << 4);
  const int vt = 4 * g + (n >> 2);                   // the lane points at this token, 4 channels from 4 (n % 4)
  const uint32_t value_at = tile_at + vt * kRowB + ((((n & 3) >> 1) ^ lat_swz(vt)) << 4) + ((n & 1) << 3);
  acc_reserve<RT>();

  int b = plan.lo.b, in_seq = plan.lo.in_seq, step0 = plan.lo.step;
  for (int j = plan.lo.tile; j < plan.hi.tile || (j == plan.hi.tile && plan.hi.step > 0); ++j, ++in_seq, step0 = 0) {
  if ((int64_t)in_seq * M >= (int64_t)load_seq(p, b).nq * p.H) {   // behind the sequence's last tile
    b = uniform(next_seq(p, b));
    in_seq = 0;
  }
  const Seq sq = load_seq(p, b);
  const int rows = sq.nq * p.H;
  const int r_tile = in_seq * M;
  const int r_last = min(r_tile + M, rows) - 1;
  const int end_max = visible(p, sq, r_last / p.H);
  const int end_min = visible(p, sq, r_tile / p.H);
  const int steps = (end_max + STEP - 1) / STEP;
  const int step1 = j == plan.hi.tile ? plan.hi.step : steps;
  const bool whole = step0 == 0 && step1 == steps;

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
  unroll<RT * kCt>([&](auto i) { acc_write<i>(v4f{0.0f, 0.0f, 0.0f, 0.0f}); });

  // The pages of 64 consecutive table entries, one a lane, from entry pbase on.
  // A wave reloads them when it comes to their end (every 64 pages).
  const int32_t* trow = p.table + (int64_t)b * p.W;
  const int last = end_max - 1;
  int pages = 0, pbase = -64;
  // The cache row of token min(tb + lane % 32, last): a token behind the last visible one is that one
  // again, so masked places hold finite values and nothing behind the sequence is read.
  auto rows_of = [&](int tb) {
    int ln = lane & 31;
    asm volatile("" : "+v"(ln));                     // so that addresses are not kept over the loop
    const uint32_t tok = (uint32_t)min(tb + ln, last);
    const int at = (int)((uint64_t)tok * p.ps_mul >> p.ps_shift);
    const int lo = uniform(at), hi = __builtin_amdgcn_readlane(at, 31);
    if (lo < pbase || hi >= pbase + 64) {
      pbase = lo;
      const int most = (int)((uint64_t)(uint32_t)last * p.ps_mul >> p.ps_shift);
      pages = clampi(trow[min(pbase + (int)(threadIdx.x & 63), most)], 0, p.P - 1);
    }
    return __shfl(pages, at - pbase) * p.ps + (int)(tok - (uint32_t)at * (uint32_t)p.ps);   // P * ps < 2^31
  };
  // 32 tokens from tb on, this wave's share of the RW waves, to LDS
  auto fetch = [&](int tb, uint8_t* to) {
    const int row = rows_of(tb);
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const uint32_t at = lds_at(to);
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < kTok / 2 / RW; ++i) {
        const int t = 2 * (i * RW + rw);
        const int64_t src = __shfl(row, t + (ln >> 5));
        dma_lanes(p.latent + src * kR + 16 * (ln & 31), at + t * kR);
      }
      const int64_t src = __shfl(row, ln & 31);
      dma_lanes(p.lat_scale + src * (kR / 128), at + kCodeB + kTok * kRopeB);
    } else {
#pragma unroll
      for (int i = 0; i < kTok / RW; ++i) {
        const int t = i * RW + rw;
        const int64_t src = __builtin_amdgcn_readlane(row, t);
        dma_row(p.latent + src * kRowB, (uint32_t)(ln ^ lat_swz(t)) << 4, at + t * kRowB);
      }
    }
#pragma unroll
    for (int i = 0; i < kTok / 8 / RW; ++i) {
      const int t = 8 * (i * RW + rw) + (ln >> 3);
      const int64_t src = __shfl(row, t);
      const int c = (ln & 7) ^ (FP8 ? 0 : rope_swz(t));
      dma_lanes(p.rope + src * kD + 8 * c, at + (FP8 ? kCodeB : kLatB) + 8 * (i * RW + rw) * kRopeB);
    }
  };
  constexpr int NB = (FP8 ? kTok / 2 / RW + 1 : kTok / RW) + kTok / 8 / RW;   // loads of a fetch
  // 16 codes to 32 bytes of bf16, exactly (power-of-two scales), at chunks 2c and 2c + 1 of token t
  auto spread = [&](int t, int c, v4u codes, float sc) {
    uint8_t* dst = tile + t * kRowB;
    *reinterpret_cast<v4u*>(dst + (((2 * c) ^ lat_swz(t)) << 4)) = __builtin_bit_cast(v4u, dequant8_bf16(codes.x, codes.y, sc));
    *reinterpret_cast<v4u*>(dst + (((2 * c + 1) ^ lat_swz(t)) << 4)) = __builtin_bit_cast(v4u, dequant8_bf16(codes.z, codes.w, sc));
  };
  // FP8, RW = 1: the tile in registers
  v4u code_reg[kTok / 2], rope_reg[kTok / 8];
  float scale_reg[kTok / 2];
  auto fetch_regs = [&](int tb) {
    const int row = rows_of(tb);
    int ln = lane;
    asm volatile("" : "+v"(ln));
#pragma unroll
    for (int i = 0; i < kTok / 2; ++i) {
      const int64_t src = __shfl(row, 2 * i + (ln >> 5));
      code_reg[i] = *reinterpret_cast<const v4u*>(p.latent + src * kR + 16 * (ln & 31));
      scale_reg[i] = p.lat_scale[src * (kR / 128) + ((ln & 31) >> 3)];
    }
#pragma unroll
    for (int i = 0; i < kTok / 8; ++i) {
      const int64_t src = __shfl(row, 8 * i + (ln >> 3));
      rope_reg[i] = *reinterpret_cast<const v4u*>(p.rope + src * kD + 8 * (ln & 7));
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  const int n_steps = step1 - step0;
  const int t_seg = step0 * STEP + tw * kTok;        // this wave's first token
  __syncthreads();                                   // the last tile's LDS is no longer read
  if constexpr (RW > 1) {
    wait_vmcnt<0>();
    for (int k = 0; k < (FP8 ? ST : ST - 1) && k < n_steps; ++k)
      fetch(t_seg + k * STEP, FP8 ? raw + k * kRawB : tile + k * kTileB);
  } else if constexpr (FP8) {
    if (t_seg < end_max && n_steps > 0) fetch_regs(t_seg);
  }
  int slot = 0;
  for (int k = 0; k < n_steps; ++k) {
    const int tb = t_seg + k * STEP;                 // first token of this wave
    uint32_t slot_at = 0;
    if constexpr (RW > 1 && !FP8) {
      if (k + ST - 1 < n_steps) wait_vmcnt<(ST - 2) * NB>();
      else wait_vmcnt<0>();
      barrier_lds();                                 // everyone's share of tile k is here, tile k - 1 is done with
      if (k + ST - 1 < n_steps) fetch(tb + (ST - 1) * STEP, tile + (slot == 0 ? ST - 1 : slot - 1) * kTileB);
      slot_at = slot * kTileB;
      slot = slot + 1 == ST ? 0 : slot + 1;
    } else if constexpr (RW > 1) {
      if (k + ST - 1 < n_steps) wait_vmcnt<(ST - 1) * NB>();
      else wait_vmcnt<0>();
      barrier_lds();
      const uint8_t* from = raw + slot * kRawB;
      int ln = lane;
      asm volatile("" : "+v"(ln));
#pragma unroll 4
      for (int i = 0; i < kTok / 2 / RW; ++i) {
        const int t = 2 * (i * RW + rw) + (ln >> 5), c = ln & 31;
        const v4u w = *reinterpret_cast<const v4u*>(from + t * kR + 16 * c);
        const float sc = reinterpret_cast<const float*>(from + kCodeB + kTok * kRopeB)[t * (kR / 128) + (c >> 3)];
        spread(t, c, w, sc);
      }
#pragma unroll
      for (int i = 0; i < kTok / 8 / RW; ++i) {
        const int t = 8 * (i * RW + rw) + (ln >> 3), c = ln & 7;
        *reinterpret_cast<v4u*>(tile + kLatB + t * kRopeB + ((c ^ rope_swz(t)) << 4)) =
            *reinterpret_cast<const v4u*>(from + kCodeB + t * kRopeB + 16 * c);
      }
      barrier_lds();
      if (k + ST < n_steps) fetch(tb + ST * STEP, raw + slot * kRawB);
      slot = slot + 1 == ST ? 0 : slot + 1;
    } else {
      if (tb >= end_max) break;                      // the other token waves have the rest
      if constexpr (FP8) {
        int ln = lane;
        asm volatile("" : "+v"(ln));
#pragma unroll
        for (int i = 0; i < kTok / 2; ++i) spread(2 * i + (ln >> 5), ln & 31, code_reg[i], scale_reg[i]);
#pragma unroll
        for (int i = 0; i < kTok / 8; ++i) {
          const int t = 8 * i + (ln >> 3);
          *reinterpret_cast<v4u*>(tile + kLatB + t * kRopeB + (((ln & 7) ^ rope_swz(t)) << 4)) = rope_reg[i];
        }
        if (k + 1 < n_steps && tb + STEP < end_max) fetch_regs(tb + STEP);
      } else {
        fetch(tb, tile);
        wait_vmcnt<0>();
      }
    }

    // scores of 32 tokens
    v4f s[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    // Operands are read kAhead fragments before their products: a wave is alone on its SIMD, so
    // nothing else covers the LDS's latency.
    v8bf x[kAhead];
    uint32_t ka = key_at + slot_at, kr = key_rope_at + slot_at, va = value_at + slot_at;
    asm volatile("" : "+v"(ka), "+v"(kr), "+v"(va));  // or the addresses below would stay in registers over the loop
    auto key = [&](auto f) {                         // fragment f: K step f / 2, tokens 16 (f % 2) ..
      constexpr int k = f / 2, tt = f % 2;
      x[f % kAhead] = k < kR / 32 ? lds_b128(ka ^ (k % 4 * 64), k / 4 * 256 + tt * 16 * kRowB)
                                  : lds_b128(kr ^ (k % 2 * 64), tt * 16 * kRopeB);
    };
    unroll<kAhead>([&](auto f) { key(f); });
    unroll<2 * kSteps>([&](auto f) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt][f % 2] = mfma_bf16(x[f % kAhead], q[rt][f / 2], s[rt][f % 2]);
      if constexpr (f + kAhead < 2 * kSteps) key(std::integral_constant<int, f + kAhead>{});
    });
    auto value = [&](auto ct) { x[ct % kAhead] = lds_tr(va ^ (ct % 8 * 32), ct / 8 * 256); };
    unroll<kAhead>([&](auto ct) { value(ct); });
    __builtin_amdgcn_sched_barrier(0);

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
      __builtin_amdgcn_sched_barrier(0);
      unroll<RT>([&](auto rt) { acc_mfma<kCt * rt + ct>(x[ct % kAhead], pr[rt]); });
      if constexpr (ct + kAhead < kCt) value(std::integral_constant<int, ct + kAhead>{});
    });
  }
  acc_settle();

  // the row's sum over the four g, then over the token waves
  float* const red = reinterpret_cast<float*>(smem);   // [4 waves][m 16, l 16], then [4 waves][512][16 rows]
  unroll<RT>([&](auto rt) {
    l[rt] += __shfl_xor(l[rt], 16);
    l[rt] += __shfl_xor(l[rt], 32);
    float part = 1.0f;                               // this token wave's weight
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
      part = m[rt] > kNegInf ? __builtin_amdgcn_exp2f(m[rt] - mt) : 0.0f;
      __syncthreads();
      float* ow = red + wave * 16 * kR;
      unroll<kCt>([&](auto ct) {
        const v4f v = acc_read<kCt * rt + ct>() * part;
#pragma unroll
        for (int e = 0; e < 4; ++e) ow[(16 * ct + 4 * g + e) * 16 + n] = v[e];
      });
      __syncthreads();
    }
    // token wave tw adds and stores the channel tiles tw kCt / TW ..
    const int r = (rw * RT + rt) * 16 + n;           // row of the tile
    if (r_tile + r <= r_last) {
      const float inv = lt > 0.0f ? 1.0f / lt : 0.0f;
      const float lse = lt > 0.0f ? mt + __builtin_log2f(lt) : kNegInf;
      const int64_t orow = (int64_t)sq.q0 * p.H + r_tile + r;
      const int64_t prow = (2 * (int64_t)w + (step0 == 0)) * M + r;
      if (tw == 0 && g == 0) {
        if (!whole) p.part_lse[prow] = lse;
        else if (p.lse) p.lse[orow] = lse * kLn2;
      }
      auto put = [&](int ct, v4f v) {
        v *= inv;
        const int c = 16 * ct + 4 * g;
        if (!whole) *reinterpret_cast<v4f*>(p.part_out + prow * kR + c) = v;
        else store4(p, orow * kR + c, v);
      };
      if constexpr (TW > 1) {
#pragma unroll 2
        for (int ct = tw * (kCt / TW); ct < (tw + 1) * (kCt / TW); ++ct) {
          v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < TW; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += red[(k * RW + rw) * 16 * kR + (16 * ct + 4 * g + e) * 16 + n];
          put(ct, v);
        }
      } else {
        unroll<kCt>([&](auto ct) { put(ct, acc_read<kCt * rt + ct>()); });
      }
    }
  });
  if (threadIdx.x == 0 && step0 == 0 && !whole) {
    // the share that finishes the tile is the first whose own end is not before, or snaps to, the tile's
    const int64_t last = ((plan.hi.end - plan.near) * plan.shares + plan.total - 1) / plan.total - 1;
    p.meta[w] = Meta{(int64_t)sq.q0 * p.H + r_tile, r_last - r_tile + 1, (int)last - w + 1};
  }
  }
}

// Joins the parts of split row tiles with weights 2^(lse_k - max).  A workgroup
// finds the split tiles (one thread per share), then takes rows of them in
// turn: two halves of 128 threads, each over every second part, 16 bytes a
// thread.  Bound by reading the parts; rows, not tiles, are dealt out, so that
// one tile in 128 parts and 128 tiles in two keep all CUs busy alike.
constexpr int kGrid = 256;    // shares: the MI355X's CUs
constexpr int kJoin = 1024;   // workgroups
__global__ void __launch_bounds__(256) join_kernel(AttnParams p, int M) {
  __shared__ Meta metas[kGrid];
  __shared__ int64_t sums[4];
  __shared__ int before[kGrid + 1];
  __shared__ float lse_max[4], weight[kGrid];
  __shared__ v4f half[128];
  const int tid = threadIdx.x;
  const Meta mine = p.meta[tid];
  metas[tid] = mine;
  int64_t all;
  const int64_t at = block_scan(mine.parts ? mine.rows : 0, sums, all);
  before[tid] = (int)at;
  if (tid == 0) before[kGrid] = (int)all;
  __syncthreads();
  for (int item = blockIdx.x; item < (int)all; item += gridDim.x) {
    int w = 0;                                       // the last share with before[w] <= item
#pragma unroll
    for (int s = kGrid / 2; s; s >>= 1)
      if (before[w + s] <= item) w += s;
    const Meta meta = metas[w];
    const int r = item - before[w];
    // part 0 is slot 1 of share w, part k slot 0 of share w + k
    auto slot = [&](int k) { return (k == 0 ? 2 * (int64_t)w + 1 : 2 * (int64_t)(w + k)) * M + r; };
    const float l = tid < meta.parts ? p.part_lse[slot(tid)] : kNegInf;
    float top = l;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    __syncthreads();                                 // the last row's weights and halves are used
    if ((tid & 63) == 0) lse_max[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(lse_max[0], lse_max[1]), fmaxf(lse_max[2], lse_max[3]));
    weight[tid] = top == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(l - top);
    __syncthreads();
    const int c = 4 * (tid & 127), odd = tid >> 7;
    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
    float sum = 0.0f;
    for (int k = odd; k < meta.parts; k += 16) {
      v4f v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)                    // parts past the last read that one again, weighing nothing
        v[u] = *reinterpret_cast<const v4f*>(p.part_out + slot(min(k + 2 * u, meta.parts - 1)) * kR + c);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float x = k + 2 * u < meta.parts ? weight[k + 2 * u] : 0.0f;
        acc += v[u] * x;
        sum += x;
      }
    }
    if (odd) half[tid & 127] = acc;
    if (tid == 128) lse_max[0] = sum;
    __syncthreads();
    if (!odd) {
      acc += half[tid];
      sum += lse_max[0];
      store4(p, (meta.row + r) * kR + c, acc * (sum > 0.0f ? 1.0f / sum : 0.0f));
      if (tid == 0 && p.lse) p.lse[meta.row + r] = sum > 0.0f ? (top + __builtin_log2f(sum)) * kLn2 : kNegInf;
    }
  }
}

// rows of an average sequence decide the tile
int tile_rows(int64_t T, int64_t H, int64_t B) {
  const int64_t per = T * H / B;
  return per >= 96 ? 128 : per >= 48 ? 64 : per >= 24 ? 32 : 16;
}

constexpr int64_t part_bytes(int m) { return (int64_t)kGrid * 2 * m * (kR + 1) * 4; }

}  // namespace

int64_t mla_attention_workspace_bytes(int64_t T, int64_t H, int64_t B) {
  return kGrid * (int64_t)sizeof(Meta) + part_bytes(tile_rows(T, H, B));
}

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
  int bits = 0;
  while ((1 << bits) < a.ps) ++bits;
  p.ps_shift = 31 + bits;
  p.ps_mul = (uint32_t)((((uint64_t)1 << p.ps_shift) + a.ps - 1) / a.ps);
  p.T = (int)a.T;
  p.H = (int)a.H;
  p.B = (int)a.B;
  p.W = (int)a.W;
  p.P = (int)a.P;
  p.ps = (int)a.ps;
  p.causal = a.causal;
  p.out_f32 = a.out_f32;
  const int m = tile_rows(a.T, a.H, a.B);
  p.meta = static_cast<Meta*>(a.workspace);
  p.part_lse = reinterpret_cast<float*>(p.meta + kGrid);
  p.part_out = p.part_lse + (int64_t)kGrid * 2 * m;
#define FP8BS_ATTN(RT_, RW_, TW_, F8_) \
  hipLaunchKernelGGL((mla_attention_kernel<RT_, RW_, TW_, F8_>), dim3(kGrid), dim3(256), 0, stream, p)
  switch (m) {
    case 128:
      if (a.fp8) FP8BS_ATTN(2, 4, 1, true);
      else FP8BS_ATTN(2, 4, 1, false);
      break;
    case 64:
      if (a.fp8) FP8BS_ATTN(2, 2, 2, true);
      else FP8BS_ATTN(2, 2, 2, false);
      break;
    case 32:   // with codes waiting in registers there is no room for two row tiles a wave
      if (a.fp8) FP8BS_ATTN(1, 2, 2, true);
      else FP8BS_ATTN(2, 1, 4, false);
      break;
    default:
      if (a.fp8) FP8BS_ATTN(1, 1, 4, true);
      else FP8BS_ATTN(1, 1, 4, false);
  }
  hipLaunchKernelGGL(join_kernel, dim3(kJoin), dim3(256), 0, stream, p, m);
#undef FP8BS_ATTN
  return hipGetLastError();
}

}  // namespace fp8bs
