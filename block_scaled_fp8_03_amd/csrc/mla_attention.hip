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
// MFMA: with 32 query rows a wave v_mfma_f32_32x32x16_bf16, with 16 rows
// v_mfma_f32_16x16x32_bf16, D = X . Y; lane (g = l / ROWS, n = l % ROWS) supplies
// row n of X and column n of Y at K values 8g .. 8g+7, and register r of its
// result is D[TS (r / 4) + 4g + r % 4][n], TS = 8 or 16.
//   scores   X = cached tokens, Y = query rows: a lane holds tokens of one query
//            row, so a row's maximum and sum are in-lane but for the g.
//   output   X = latent channels (transposed reads), Y = the probabilities: a
//            lane's eight scores r are taken as its K values 8g + r, so they go from
//            the score's registers to the operand without crossing lanes, and the
//            latents' tokens are read in that order by two 4-token transposed LDS
//            reads.
//
// A wave carries ROWS query rows (Q in registers) over 32 cached tokens at a
// time; RW waves take different rows of the same tokens and TW waves different
// tokens of the same rows.
//
// What bounds it.  A cached token of 1152 (bf16) or 656 (FP8) bytes costs 2176
// flops a row: the matrix cores bound 128 rows and more a token, HBM 16.  A row
// tile holds 288 KB of Q and accumulators at 128 rows, which is why a workgroup
// has a CU to itself, one wave a SIMD, and hides latency by reading ahead.
// Measured on an MI355X (copies reach 4.9 TB/s, large bf16 products 1.4 to 1.6
// PFLOP/s):
//   128 rows  512 new tokens on 8192, 128 heads: 890 to 960 us, 1.18 to 1.27 PFLOP/s; matrix
//             cores busy 67% of the cycles, at 1.7 to 2.0 GHz.  1.75 us a step of 32 tokens with
//             bf16, 1.85 with FP8; the products alone are 1.1 us.
//   64 rows   32 x 4096 tokens, 128 heads: 66 to 71 us with the join, 40 of them the loop, at 3.8 TB/s
//             with each token read by two tiles
//   16 rows   128 sequences of up to 8192 tokens, 16 heads, FP8: 98 to 101 us, 4.1 TB/s
//   least     one token, 16 heads, 500 cached: 19 us; 12 of them this kernel (plan 2, pages, Q
//             and tokens 4, a step of 128 tokens 1.7, the four token waves' sum 3.1), the join 5
#include <algorithm>
#include <cmath>
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
constexpr int kRopeB = kD * 2;
// 32 tokens in LDS: four blocks of 8 tokens, each nine groups (eight of latents,
// one rotated) of 128 bytes a token.  A group is one load instruction, and the
// groups of a token are 128 bytes apart in memory and 1024 in LDS.
constexpr int kGroupB = 8 * 128;
constexpr int kBlockB = 9 * kGroupB;
constexpr int kTileB = 4 * kBlockB;     // 36,864 bytes
// FP8: 8 tokens as they come: four groups of codes, the rotated group (with PIPE it goes to its
// place in the tile at once), four scales a token (twice)
template <bool PIPE>
constexpr int raw_bytes() { return (PIPE ? 4 : 5) * kGroupB + 256; }
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
  float scale2;             // |scale| * log2(e)
  uint32_t flip;            // scale < 0: the sign bits of two bf16, put on Q
  uint32_t ps_mul;          // tok / ps = tok * ps_mul >> ps_shift for tok < 2^31
  int ps_shift;
  // workspace: [grid] Meta, then [grid][2][M] lse (base 2), then [grid][2][M][512] normalised output parts
  struct Meta* meta;
  float* part_lse;
  float* part_out;
  int T, H, B, W, P, ps;
  int longest;              // tokens of a sequence: W * ps, and so few that positions some tiles ahead fit 32 bits
  int causal, out_f32;
};

// what a workgroup leaves for the join: the row tile that it begins and does not finish
struct Meta {
  int64_t row;      // its first row of [T * H]
  int rows, parts;  // parts = 0: none.  Part 0 is this workgroup's, part k the k-th next one's.
};

// The 16-byte chunk c of token t sits in group c / 8 at place (c % 8) ^ swz(t): a
// linear map of the token's bits chosen for the LDS's rule (a b128 read is
// served in four cycles of the 16 lanes of a half-wave with equal parity of
// lane bits 2..4, a b64 read by half-waves, over 64 banks), under which both the
// score reads and the transposed reads touch 16 distinct slots of 16 bytes a cycle.
template <int ROWS>
__device__ __forceinline__ int swz(int t) {
  const int t1 = (t >> 1) & 1, t2 = (t >> 2) & 1, t3 = (t >> 3) & 1;
  return ROWS == 32 ? t1 << 2 | t3 << 1 | t2 : t1 << 2 | t2 << 1 | t2;
}

typedef float v16f __attribute__((ext_vector_type(16)));
__device__ __forceinline__ v4f mfma_bf16(v8bf x, v8bf y, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
}
__device__ __forceinline__ v16f mfma_bf16(v8bf x, v8bf y, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t lds_at(const void* q) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)q;
}
__device__ __forceinline__ v8bf lds_b128(uint32_t at, int off) {
  return __builtin_bit_cast(v8bf, *((const lds_v4u*)(uintptr_t)at + off / 16));
}
// 4 tokens x 16 channels a quarter-wave, transposed, twice
__device__ __forceinline__ v8bf lds_tr(uint32_t at0, int off0, uint32_t at1, int off1) {
  typedef short v8s __attribute__((ext_vector_type(8)));
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)at0 + off0 / 8);
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)at1 + off1 / 8);
  return __builtin_bit_cast(v8bf, (v8s)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The output accumulators: AGPRs 0 .. 8 ROWS - 1, named in the instructions
// below; 256 a lane with 32 rows.  Left to the compiler they would be VGPRs (the
// rare rescale is VALU work, which cannot take AGPRs), and with Q's registers
// that spilled 230 of them to memory.  The source is built so that the
// compiler itself puts nothing into AGPRs (its own MFMAs in the VGPR form, and
// less than 256 VGPRs live); the build refuses a listing where it does.
// Wait states: a VALU result may be an MFMA operand two instructions later, which
// the build checks too; an MFMA's result may be read by another kind of
// instruction 19 cycles later, for which acc_settle stands.
template <int ROWS, int T>
__device__ __forceinline__ void acc_mfma(v8bf x, v8bf y) {
  if constexpr (ROWS == 32)
    asm volatile("v_mfma_f32_32x32x16_bf16 a[%0:%1], %2, %3, a[%0:%1]"
                 :: "n"(16 * T), "n"(16 * T + 15), "v"(x), "v"(y));
  else
    asm volatile("v_mfma_f32_16x16x32_bf16 a[%0:%1], %2, %3, a[%0:%1]"
                 :: "n"(4 * T), "n"(4 * T + 3), "v"(x), "v"(y));
}
__device__ __forceinline__ void acc_settle() { asm volatile("s_nop 15\n\ts_nop 15"); }
__device__ __forceinline__ void operands_settle() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 1");
}
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
// Four e4m3 codes times a power-of-two scale, exactly, in bf16: the instruction takes the scale's
// exponent (checked over all codes and the scales 2^-100 .. 2^100).
__device__ __forceinline__ v2u codes4_bf16(uint32_t codes, float scale) {
  return v2u{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, false)),
             __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, true))};
}

// calls f with the constants 0 .. N-1
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unroll(const F& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unroll<N, I + 1>(f);
  }
}
// tells the compiler how many AGPRs a kernel takes
template <int ROWS>
__device__ __forceinline__ void acc_reserve() {
  if constexpr (ROWS == 16) asm volatile("" ::: "a127");
  else asm volatile("" ::: "a255");
}

// A lane's scores of 32 tokens: number e is that of token TS (e / 4) + 4g + e % 4
template <int ROWS>
struct Scores;
template <>
struct Scores<32> {
  static constexpr int N = 16, TS = 8;
  v16f v;
  __device__ void clear() {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = 0.0f;
  }
  template <int E> __device__ float get() const { return v[E]; }
  template <int E> __device__ void set(float x) { v[E] = x; }
};
template <>
struct Scores<16> {
  static constexpr int N = 8, TS = 16;
  v4f v[2];
  __device__ void clear() { v[0] = v[1] = v4f{0.0f, 0.0f, 0.0f, 0.0f}; }
  template <int E> __device__ float get() const { return v[E / 4][E % 4]; }
  template <int E> __device__ void set(float x) { v[E / 4][E % 4] = x; }
};

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
  s.len = clampi(p.lens[b], 0, p.longest);
  return s;
}

// cached tokens that query token i of a sequence sees
__device__ __forceinline__ int visible(const AttnParams& p, const Seq& s, int i) {
  return p.causal ? clampi(s.len - s.nq + i + 1, 0, s.len) : s.len;
}

// Direct global -> LDS loads of 16 (4) bytes a lane: lane i's bytes at `at` + OFF
// land at lds + 16 i (4 i).  The instruction adds OFF to both addresses.  In
// assembly, so that the compiler does not make every LDS read wait for all of
// them; completion is awaited with wait_vmcnt.
template <int OFF>
__device__ __forceinline__ void dma_b128(const void* at, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off offset:%2"
               :: "s"(__builtin_amdgcn_readfirstlane(lds - OFF)), "v"(at), "n"(OFF) : "memory", "m0");
}
__device__ __forceinline__ void dma_b32(const void* at, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
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

// exclusive prefix sum over the workgroup's WAVES waves; total gets the sum
template <int WAVES = 4>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sums, int64_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t x = wave_scan(v);
  __syncthreads();
  if (lane == 63) sums[wave] = x;
  __syncthreads();
  int64_t base = 0;
  total = 0;
#pragma unroll
  for (int k = 0; k < WAVES; ++k) {
    if (k < wave) base += sums[k];
    total += sums[k];
  }
  return base + x - v;
}

// ---------------------------------------------------------------------------
// The work split.  The grid is one workgroup per CU, whatever the batch.  The
// row tiles of all sequences, in order, cost start_cost + (steps of 32 TW cached
// tokens) each; the sum of the costs is cut into equal shares, and workgroup w
// works through share w: the end of one tile's tokens, whole tiles, the
// beginning of another's.  So long and short sequences, few rows and many, all
// fill the card evenly, from lengths that only the device knows.  A tile that
// several workgroups share is joined by join_kernel from at most two parts per
// workgroup.  Every workgroup computes the split itself: two prefix sums, over
// the sequences (row tiles) and over the row tiles (costs).
// ---------------------------------------------------------------------------
// It takes about 2 us of each workgroup: the batch's lengths read, two prefix sums, the search.
// A tile's queries and output, in steps.  Measured with 2, 4 and 6 (24 sequences of up to 2777 tokens, 61
// new each, us): 16 heads 88.4 / 89.1 / 93.1, 128 heads 401 / 392 / 394.  16 rows' steps are of 128
// tokens: 91 single tokens on up to 4319, 16 heads, with 2 and 4 69.4 / 70.9.
template <int M>
constexpr int start_cost() { return M == 16 ? 2 : 4; }
// A share is no smaller, so that short work is not cut to pieces: 128 cached tokens with 128 rows a
// tile (a step is 32), one step of 128 with 16 rows.
template <int M>
constexpr int least() { return M == 128 ? 4 : M == 64 ? 2 : 1; }
// A cut this near a tile's edge moves to it: a split costs the writing and
// reading of M rows of float32 twice, about M / 16 steps' time.  (Twice as near loses more
// balance than it saves: the 16 heads above 89 / 103.)
template <int M>
__device__ __forceinline__ int slack(int64_t total, int shares) { return (int)min((int64_t)(M / 16), total / shares / 2); }

struct Cut {          // a place between two steps
  int tile;           // row tile of the batch
  int b, in_seq;      // its sequence, its index there
  int step;
  int64_t end;        // cuts from this cost on snap to the tile's end
};

// values that all lanes share, moved to scalar registers
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}
__device__ __forceinline__ Cut uniform(const Cut& c) {
  return Cut{uniform(c.tile), uniform(c.b), uniform(c.in_seq), uniform(c.step), uniform(c.end)};
}

constexpr int kSeqs = 8192;  // sequences whose lengths the plan holds in LDS

template <int M, int STEP>
struct Plan {
  Cut lo, hi;
  int64_t total;
  int shares;

  static __device__ int tile_steps(const AttnParams& p, const Seq& s, int in_seq) {
    const int r = (int)min((int64_t)(in_seq + 1) * M, (int64_t)s.nq * p.H) - 1;
    return (visible(p, s, r / p.H) + STEP - 1) / STEP;
  }
  // A short chunk's tiles all cost what its last does (at most a seventh more than they
  // take, and a step: its first token sees over 7/8 of the sequence): equal costs, and cuts
  // fall on the tiles' edges where their number allows.
  static __device__ int tile_cost(const AttnParams& p, const Seq& s, int in_seq) {
    return start_cost<M>() + (s.nq <= s.len / 8 ? (s.len + STEP - 1) / STEP : tile_steps(p, s, in_seq));
  }

  static constexpr int kBytes = 256 + 4 * (kSeqs + 4) + (int)sizeof(Seq) * kSeqs;
  // false: this workgroup has no share
  __device__ bool make(const AttnParams& p, int w, uint8_t* smem) {
    int64_t* sums = reinterpret_cast<int64_t*>(smem);
    Cut* cut = reinterpret_cast<Cut*>(smem + 64);
    int* first = reinterpret_cast<int*>(smem + 256);       // [B + 1] row tiles before each sequence
    Seq* seq = reinterpret_cast<Seq*>(smem + 256 + 4 * (kSeqs + 4));
    const int tid = threadIdx.x;
    const int per_b = (p.B + 255) / 256;
    const int b0 = min(tid * per_b, p.B), b1 = min(b0 + per_b, p.B);
    int64_t mine = 0, sum;
    for (int b = b0; b < b1; ++b) {
      seq[b] = load_seq(p, b);
      mine += ((int64_t)seq[b].nq * p.H + M - 1) / M;
    }
    int64_t at = block_scan(mine, sums, sum);
    // a cu_q that decreases lays sequences over each other: such a batch is left undone when its rows are more
    // than there are, so that the counts stay in range and the work bounded
    if (sum > (int64_t)p.T * p.H / M + p.B) return false;
    const int tiles = (int)sum;
    for (int b = b0; b < b1; ++b) {
      first[b] = (int)at;
      at += ((int64_t)seq[b].nq * p.H + M - 1) / M;
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
    for (int t = t0; t < t1; ++t) {
      while (t >= first[b + 1]) ++b;
      mine += tile_cost(p, seq[b], t - first[b]);
    }
    int64_t base = block_scan(mine, sums, total);
    total = uniform(total);
    shares = (int)max((int64_t)1, min((int64_t)gridDim.x, total / least<M>()));
    if (w >= shares || total == 0) return false;

    const int near = slack<M>(total, shares);
    const int64_t want[2] = {total * w / shares, total * (w + 1) / shares};
    if (t1 == tiles && t0 < t1 && want[1] == total) cut[1] = Cut{tiles, p.B, 0, 0, total};
    if (t0 < t1 && ((want[0] >= base && want[0] < base + mine) || (want[1] >= base && want[1] < base + mine))) {
      b = bs;
      for (int t = t0; t < t1; ++t) {
        while (t >= first[b + 1]) ++b;
        const int in_seq = t - first[b], c = tile_cost(p, seq[b], in_seq);
        const int done = min(c - near, start_cost<M>() + tile_steps(p, seq[b], in_seq));
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (want[k] >= base && want[k] < base + c) {
            const int at = (int)(want[k] - base);
            // (tile t + 1 may be the next sequence's first: the share that begins there looks)
            if (at <= start_cost<M>() + near) cut[k] = Cut{t, b, in_seq, 0, base + done};
            else if (at >= done) cut[k] = Cut{t + 1, b, in_seq + 1, 0, base + done};
            else cut[k] = Cut{t, b, in_seq, at - start_cost<M>(), base + done};
          }
        base += c;
      }
    }
    __syncthreads();
    lo = uniform(cut[0]);
    hi = uniform(cut[1]);
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

// LDS.  One token wave's tiles: with PIPE (RW = 4) a ring of four, or three and two
// stages of codes for FP8; with RW = 2 two, or one and two stages of codes; with
// RW = 1 one (FP8: the codes wait in registers).  A wave makes bf16 of the codes
// that it loaded itself.
template <int RW, bool FP8>
constexpr int tiles() { return RW == 4 ? (FP8 ? 3 : 4) : RW == 2 && !FP8 ? 2 : 1; }
template <int RW, bool FP8>
constexpr int raws() { return !FP8 || RW == 1 ? 0 : 2; }
template <int ROWS, int RW, int TW, bool FP8>
constexpr int lds_bytes() {
  const int n = TW * (tiles<RW, FP8>() * kTileB + raws<RW, FP8>() * 4 * raw_bytes<RW == 4>()) + (RW == 4 ? 4 * 4 * 1024 : 0);
  return TW > 1 ? std::max(n, 4 * ROWS * (kR / (ROWS / 16)) * 4) : n;   // the token waves' accumulators meet here
}

template <int ROWS, int RW, int TW, bool FP8>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
mla_attention_kernel(AttnParams p) {
  constexpr int M = ROWS * RW, STEP = kTok * TW;
  constexpr bool WIDE = ROWS == 32, PIPE = RW == 4;
  constexpr int NT = tiles<RW, FP8>(), NR = raws<RW, FP8>(), kRawB = raw_bytes<PIPE>();
  constexpr int NSUB = 4 / RW;                       // blocks of 8 tokens that a wave loads of 32
  constexpr int CH = 8 * 64 / ROWS;                  // channels of a K step of the scores
  constexpr int QN = (kR + kD) / CH;                 // K steps
  constexpr int QS = PIPE && WIDE ? kR / CH : QN;          // those whose Q is in registers; PIPE: the rotated ones are in LDS
  // Fragments read ahead of their products: the LDS's latency in products of 32 cycles, or of 16
  // (16 rows: 6 ahead left the waves waiting half the time; with the codes in registers there is no room)
  constexpr int kAhead = WIDE || (FP8 && RW == 1) ? 6 : 12;
  constexpr int NV = 32;                             // fragments of the latents as values
  constexpr int NF = 36;                             // fragments of the latents as keys
  constexpr int GS = Scores<ROWS>::TS, NG = kR / GS; // accumulators: NG groups of 4 channels from GS i + 4 g
  static_assert(RW * TW == 4 && lds_bytes<ROWS, RW, TW, FP8>() <= 160 * 1024 &&
                Plan<M, STEP>::kBytes <= lds_bytes<ROWS, RW, TW, FP8>(), "layout");
  static_assert(NF % kAhead == 0 && kAhead % 2 == 0, "the two streams of fragments share x");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[lds_bytes<ROWS, RW, TW, FP8>()];
  const int lane = threadIdx.x & 63;
  const int n = lane % ROWS, g = lane / ROWS;
  const int wave = uniform((int)threadIdx.x >> 6);
  const int rw = wave % RW, tw = wave / RW;
  const uint32_t tile_at = lds_at(smem) + tw * NT * kTileB;                             // this token wave's tiles
  const uint32_t raw_at = lds_at(smem) + TW * NT * kTileB + wave * NR * NSUB * kRawB;   // this wave's codes
  const uint32_t rest_at = lds_at(smem) + NT * kTileB + 4 * NR * kRawB + wave * 4096;   // PIPE: its Q, [4][lane] 16 bytes

  // neighbouring shares on one XCD (workgroups go round the eight): they often stream the same tokens
  const int w = gridDim.x % 8 == 0 ? (blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8 : blockIdx.x;
  if (threadIdx.x == 0) p.meta[w].parts = 0;
  Plan<M, STEP> plan;
  if (!plan.make(p, w, smem)) return;

  // The operand reads' addresses in a tile.  A chunk's swizzle touches the low three bits of its
  // index alone and by exclusive or, so K step s (2 or 4 chunks on) has 16 (its chunk % 8) xored in and
  // 1024 (its chunk / 8) added, and so have the channel tiles.
  const uint32_t key_at = tile_at + n / 8 * kBlockB + n % 8 * 128 + ((g ^ swz<ROWS>(n)) << 4);
  uint32_t value_at;
  {
    const int q = lane & 15, tok = 4 * g + (q >> 2), c = (WIDE ? (lane >> 4 & 1) * 2 : 0) + ((q & 3) >> 1);
    value_at = tile_at + tok / 8 * kBlockB + tok % 8 * 128 + ((c ^ swz<ROWS>(tok)) << 4) + ((q & 1) << 3);
  }
  acc_reserve<ROWS>();

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

  wait_vmcnt<0>();
  __syncthreads();                                   // the last tile's LDS is no longer read or written

  float m = kNegInf, l = 0.0f;
  unroll<2 * ROWS>([&](auto i) { acc_write<i>(v4f{0.0f, 0.0f, 0.0f, 0.0f}); });

  // The pages of 64 consecutive table entries, one a lane, from entry pbase on.
  // A wave reloads them when it comes to their end (every 64 pages).
  const int32_t* trow = p.table + (int64_t)b * p.W;
  const int last = end_max - 1;
  int pages = 0, pbase = -64;
  // 8 tokens from tb on to a block of LDS: token lane / 8, 16 bytes from 16 (lane % 8) of each group.
  // A token behind the last visible one is that one again, so masked places hold finite values and
  // nothing behind the sequence is read.
  struct From {
    const uint8_t* lat;
    const uint16_t* rope;
    const float* scale;
  };
  auto find = [&](int tb, int sub) {
    int ln = lane;
    asm volatile("" : "+v"(ln));                     // so that addresses are not kept over the loop
    const uint32_t tok = (uint32_t)min(tb + 8 * sub + (ln >> 3), last);
    const int at = (int)((uint64_t)tok * p.ps_mul >> p.ps_shift);
    const int lo = uniform(at), hi = __builtin_amdgcn_readlane(at, 63);
    if (lo < pbase || hi >= pbase + 64) {
      pbase = lo;
      const int most = (int)((uint64_t)(uint32_t)last * p.ps_mul >> p.ps_shift);
      pages = clampi(trow[min(pbase + ln, most)], 0, p.P - 1);
    }
    // P * ps < 2^31
    const int64_t row = __shfl(pages, at - pbase) * p.ps + (int)(tok - (uint32_t)at * (uint32_t)p.ps);
    const int c = (ln & 7) ^ swz<ROWS>(8 * sub + (ln >> 3));   // the chunk for this lane's place
    From f;
    f.lat = p.latent + row * (FP8 ? kR : 2 * kR) + 16 * (FP8 ? ln & 7 : c);
    f.rope = p.rope + row * kD + 8 * (FP8 && !PIPE ? ln & 7 : c);
    f.scale = FP8 ? p.lat_scale + row * (kR / 128) + (ln & 3) : nullptr;
    return f;
  };
  constexpr int NL = FP8 ? 6 : 9;                    // loads of a block
  // load i of a block; `to` is the block in the tile, `codes` (FP8) the block's stage
  auto ask = [&](const From& f, uint32_t to, uint32_t codes, auto i) {
    constexpr int rope = FP8 ? 4 : 8;
    if constexpr (i < rope) dma_b128<128 * i>(f.lat, (FP8 ? codes : to) + i * kGroupB);
    else if constexpr (i == rope) dma_b128<0>(f.rope, FP8 && !PIPE ? codes + 4 * kGroupB : to + 8 * kGroupB);
    else dma_b32(f.scale, codes + (PIPE ? 4 : 5) * kGroupB);
  };
  // this wave's blocks of 32 tokens, to a tile and (FP8) a stage of the wave's codes
  auto fetch = [&](int tb, uint32_t to, uint32_t codes) {
#pragma unroll
    for (int i = 0; i < NSUB; ++i) {
      const int sub = rw * NSUB + i;
      const From f = find(tb, sub);
      unroll<NL>([&](auto u) { ask(f, to + sub * kBlockB, codes + i * kRawB, u); });
    }
  };
  // Codes to bf16, exactly (power-of-two scales): the 16 codes of group i that this lane loaded, to
  // chunks 2c and 2c + 1 of its token, c = lane % 8 + 8 i
  auto spread = [&](int sub, int i, v4u codes, float sc, uint32_t to) {
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const int t = ln >> 3, c = 2 * (ln & 3);
    const uint32_t at = to + sub * kBlockB + (2 * i + ((ln & 7) >> 2)) * kGroupB + t * 128;
    const int x = swz<ROWS>(8 * sub + t);
    const v2u d0 = codes4_bf16(codes.x, sc), d1 = codes4_bf16(codes.y, sc), d2 = codes4_bf16(codes.z, sc), d3 = codes4_bf16(codes.w, sc);
    *(lds_v4u*)(uintptr_t)(at + ((c ^ x) << 4)) = v4u{d0.x, d0.y, d1.x, d1.y};
    *(lds_v4u*)(uintptr_t)(at + (((c + 1) ^ x) << 4)) = v4u{d2.x, d2.y, d3.x, d3.y};
  };
  auto spread_rope = [&](int sub, v4u v, uint32_t to) {
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const int t = ln >> 3;
    *(lds_v4u*)(uintptr_t)(to + sub * kBlockB + 8 * kGroupB + t * 128 + (((ln & 7) ^ swz<ROWS>(8 * sub + t)) << 4)) = v;
  };
  // piece i < 5 of a block's codes from LDS: a group, or the rotated one
  auto spread_raw = [&](int sub, auto i, uint32_t from, uint32_t to) {
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const v4u v = *(const lds_v4u*)(uintptr_t)(from + i * kGroupB + ln * 16);
    if constexpr (i < 4) {
      typedef const __attribute__((address_space(3))) float lds_f;
      spread(sub, i, v, *(lds_f*)(uintptr_t)(from + 5 * kGroupB + (ln >> 3) * 32 + i * 4), to);
    } else {
      spread_rope(sub, v, to);
    }
  };
  // PIPE: the same in 20 pieces of a few instructions: group i is read in piece 4 i, and converted and
  // written in the pieces 4 i + 5 .. + 7, when it has come
  v4u some_codes[2], some_bf16[2];
  float some_scale[2];
  uint32_t codes_from = 0, scales_from = 0, bf16_to = 0;
  auto spread_at = [&](uint32_t from, uint32_t to) {
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const int t = ln >> 3, c = 2 * (ln & 3);
    codes_from = from + ln * 16;
    scales_from = from + 4 * kGroupB + t * 32;
    bf16_to = to + rw * kBlockB + ((ln & 7) >> 2) * kGroupB + t * 128 + ((c ^ swz<ROWS>(8 * rw + t)) << 4);
  };
  auto spread_bit = [&](auto u) {
    constexpr int i = u / 4, k = u % 4;
    typedef const __attribute__((address_space(3))) float lds_f;
    if constexpr (k == 0 && i < 4) {
      some_codes[i % 2] = *((const lds_v4u*)(uintptr_t)codes_from + i * 64);
      some_scale[i % 2] = *((lds_f*)(uintptr_t)scales_from + i);
    } else if constexpr (i > 0 && k > 0 && k < 3) {
      const v4u w = some_codes[(i - 1) % 2];
      const v2u a = codes4_bf16(w[2 * k - 2], some_scale[(i - 1) % 2]), c = codes4_bf16(w[2 * k - 1], some_scale[(i - 1) % 2]);
      some_bf16[k - 1] = v4u{a.x, a.y, c.x, c.y};
    } else if constexpr (i > 0 && k == 3) {
      *((lds_v4u*)(uintptr_t)bf16_to + (i - 1) * 2 * 64) = some_bf16[0];
      *((lds_v4u*)(uintptr_t)(bf16_to ^ 16) + (i - 1) * 2 * 64) = some_bf16[1];
    }
  };
  // FP8, RW = 1: the codes in registers
  v4u code_reg[16], rope_reg[4];
  float scale_reg[16];
  auto fetch_regs = [&](int tb) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const From f = find(tb, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        code_reg[4 * s + i] = *reinterpret_cast<const v4u*>(f.lat + 128 * i);
        scale_reg[4 * s + i] = (f.scale - (lane & 3))[i];
      }
      rope_reg[s] = *reinterpret_cast<const v4u*>(f.rope);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  const int n_steps = step1 - step0;
  const int t_seg = step0 * STEP + tw * kTok;        // this wave's first token
  // the first tokens are on their way before Q
  if constexpr (PIPE) {
    if (n_steps > 0)
      for (int k = 0; k < (FP8 ? 2 : NT - 1); ++k) fetch(t_seg + k * STEP, tile_at + k * kTileB, raw_at + (FP8 ? k * kRawB : 0));
  } else if constexpr (RW > 1) {
    for (int k = 0; k < (FP8 ? 2 : 1) && k < n_steps; ++k) fetch(t_seg + k * STEP, tile_at, raw_at + k * NSUB * kRawB);
  } else if (t_seg < end_max && n_steps > 0) {
    if constexpr (FP8) fetch_regs(t_seg);
    else fetch(t_seg, tile_at, 0u);
  }

  // this lane's query row: its operands, and the tokens it sees
  v8bf q[QS];
  int end;
  {
    int ln = lane;
    asm volatile("" : "+v"(ln));                     // addresses made here, and in the end, do not stay in registers
    const int r = min(r_tile + rw * ROWS + ln % ROWS, r_last);
    const int i = r / p.H, h = r - i * p.H;
    end = visible(p, sq, i);
    const uint16_t* ql = p.q_lat + (sq.q0 + i) * p.ldq_t + h * p.ldq_h + 8 * (ln / ROWS);
    const uint16_t* qr = p.q_rope + (sq.q0 + i) * p.ldr_t + h * p.ldr_h + 8 * (ln / ROWS);
#pragma unroll
    for (int s = 0; s < QN; ++s) {
      v4u v = *reinterpret_cast<const v4u*>(s < kR / CH ? ql + CH * s : qr + CH * s - kR);
      v ^= p.flip;
      if (s < QS) q[s] = __builtin_bit_cast(v8bf, v);
      else *((lds_v4u*)(uintptr_t)(rest_at + ln * 16) + (s - QS) * 64) = v;
    }
  }

  // Operands are read kAhead fragments before their products: a wave is alone on its SIMD, so
  // nothing else covers the LDS's latency.
  v8bf x[kAhead];
  Scores<ROWS> s;
  v8bf pr[WIDE ? 2 : 1];
  uint32_t ka[WIDE ? 4 : 2], va[4];
  // the tile's addresses, opaque, or those made from them would stay in registers over the loop
  auto keys_at = [&](uint32_t off) {
    uint32_t at = key_at + off;
    asm volatile("" : "+v"(at));
#pragma unroll
    for (int i = 0; i < (WIDE ? 4 : 2); ++i) ka[i] = at ^ (i * (WIDE ? 32 : 64));
  };
  auto values_at = [&](uint32_t off) {
    uint32_t at = value_at + off;
    asm volatile("" : "+v"(at));
#pragma unroll
    for (int i = 0; i < 4; ++i) va[i] = at ^ (i * 32);
  };
  // fragment f of the keys: WIDE: K step f, 32 tokens; else K step f / 2, 16 tokens from 16 (f % 2)
  auto key = [&](auto f) {
    if constexpr (WIDE) x[f % kAhead] = lds_b128(ka[f % 4], f / 4 * kGroupB);
    else x[f % kAhead] = lds_b128(ka[f / 2 % 2], f / 4 * kGroupB + f % 2 * 2 * kBlockB);
  };
  // and its product; the rotated part of Q comes from LDS two steps before it is needed
  v8bf qr[PIPE ? 4 : 1];
  auto score = [&](auto f, Scores<ROWS>& to) {
    if constexpr (WIDE) {
      if constexpr (f < QS) to.v = mfma_bf16(x[f % kAhead], q[f], to.v);
      else to.v = mfma_bf16(x[f % kAhead], qr[(f - QS) % 4], to.v);
      if constexpr (PIPE && f + 4 >= QS && f < QS) qr[(f + 4 - QS) % 4] = lds_b128(rest_at + lane * 16, (f + 4 - QS) * 1024);
    } else {
      to.v[f % 2] = mfma_bf16(x[f % kAhead], q[f / 2], to.v[f % 2]);
    }
  };
  // fragment f of the values: WIDE: 32 channels from 32 (f / 2), 16 tokens from 16 (f % 2); else 16
  // channels from 16 f, 32 tokens
  auto read_value = [&](auto f) {
    if constexpr (WIDE) {
      constexpr int off = f / 4 * kGroupB + f % 2 * 2 * kBlockB;
      return lds_tr(va[f / 2 % 2 * 2], off, va[f / 2 % 2 * 2 + 1], off + kBlockB);
    } else {
      constexpr int off = f / 4 * kGroupB;
      return lds_tr(va[f % 4], off, va[f % 4], off + 2 * kBlockB);
    }
  };
  auto value = [&](auto f) { x[f % kAhead] = read_value(f); };
  auto product = [&](auto f) {
    if constexpr (WIDE) acc_mfma<ROWS, f / 2>(x[f % kAhead], pr[f % 2]);
    else acc_mfma<ROWS, f>(x[f % kAhead], pr[0]);
  };
  // Tiles that some row does not see whole: the scores' masked places, and tokens that are not finite.
  // A token that some row of the tile does not see may hold infinities or NaN, which a probability of 0
  // does not take out of the product.  Every row's score of it is then not finite either, so the
  // masked scores tell (`hidden`), and what is not finite in the values becomes 0.  A row that sees such a
  // token has NaN in its sum, unless the score is -inf (`low`): its probability is 0, and 0 times an infinity
  // is NaN in that channel alone, which is put into the accumulators before.
  auto mask = [&](int tb, float& hidden, float& low) {   // hidden becomes NaN, low -inf
    if (tb + kTok <= end_min) return;
    unroll<Scores<ROWS>::N>([&](auto e) {
      const float v = s.template get<e>();
      const bool sees = tb + GS * (e / 4) + 4 * g + e % 4 < end;
      hidden = __builtin_fmaf(sees ? 0.0f : v, 0.0f, hidden);
      low = fminf(low, sees ? v : 0.0f);
      s.template set<e>(sees ? v : kNegInf);
    });
  };
  // NaN into the accumulators of the channels where a token that the row sees with a score of -inf holds
  // what is not finite: 2^127.99 squared overflows to inf, and inf - inf is NaN
  auto mark = [&](int tb) {
    v4u u[2];
    unroll<Scores<ROWS>::N>([&](auto e) {
      const bool in = tb + GS * (e / 4) + 4 * g + e % 4 < end && s.template get<e>() == kNegInf;
      const uint32_t one = in ? e % 2 ? 0x7F7F0000u : 0x7F7Fu : 0u;
      if constexpr (e % 2 == 0) u[e / 8][e % 8 / 2] = one;
      else u[e / 8][e % 8 / 2] |= one;
    });
    unroll<Scores<ROWS>::N / 8>([&](auto k) { pr[k] = __builtin_bit_cast(v8bf, u[k]); });
    unroll<NV>([&](auto f) {
      v4u v = __builtin_bit_cast(v4u, read_value(f));
#pragma unroll
      for (int d = 0; d < 4; ++d)
        v[d] = ((v[d] & 0x7F80u) == 0x7F80u ? 0x7F7Fu : 0u) | ((v[d] & 0x7F800000u) == 0x7F800000u ? 0x7F7F0000u : 0u);
      const v8bf plus = __builtin_bit_cast(v8bf, v), minus = __builtin_bit_cast(v8bf, v ^ (v << 1 & 0x80008000u));
      operands_settle();
      acc_mfma<ROWS, WIDE ? f / 2 : f>(plus, pr[WIDE ? f % 2 : 0]);
      acc_mfma<ROWS, WIDE ? f / 2 : f>(minus, pr[WIDE ? f % 2 : 0]);
    });
  };
  auto clear = [&](uint32_t tile) {
    int ln = lane;
    asm volatile("" : "+v"(ln));
    uint32_t at = tile + ln * 16;
#pragma unroll 1
    for (int i = 0; i < 4 * 8; ++i) {
      v4u v = *(const lds_v4u*)(uintptr_t)at;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        if ((v[d] & 0x7F80u) == 0x7F80u) v[d] &= 0xFFFF0000u;
        if ((v[d] & 0x7F800000u) == 0x7F800000u) v[d] &= 0xFFFFu;
      }
      *(lds_v4u*)(uintptr_t)at = v;
      at += i % 8 == 7 ? 2 * kGroupB : kGroupB;      // past the rotated group
    }
  };
  // all of it for step k, its tokens from tb on (values_at is set); true if the tile's values changed.  The other
  // row waves' scores and marks are of the values as they came, hence the barrier; their products may
  // take the cleared values or not: theirs are rows that do not see the token, or have NaN by now.
  // (No bf16 of a code is infinite, and a NaN gives no score of -inf: FP8 has nothing to mark.)
  auto hide = [&](int k, int tb, uint32_t tile) {
    float hidden = 0.0f, low = 0.0f;
    mask(tb, hidden, low);
    if (end_min == end_max || (step0 + k + 1) * STEP <= end_min) return false;
    if constexpr (!FP8)
      if (__any(low == kNegInf)) mark(tb);
    if constexpr (RW > 1 && !(FP8 && PIPE)) barrier_lds();   // (PIPE: the scores are a barrier ago)
    if (!__any(hidden != hidden)) return false;
    clear(tile);
    return true;
  };
  // Scores to probabilities in kSoft pieces that fit beside a matrix instruction: the maximum of four
  // scores; the check of it; one probability; eight of them packed.
  // The probabilities are rounded to bf16 (half a step, 2^-8 of each, with its own sign): the product takes both
  // operands in 16 bits, and a second product with what the rounding left would lengthen the matrix-bound
  // loop by nearly half.  It is the largest error here: relative to 64 bits, 0.0017 to 0.0022 with a bf16
  // output, which alone is 0.0017.  The sum l has them unrounded, in float32.
  constexpr int NS = Scores<ROWS>::N, kSoft = NS / 4 + 1 + NS + NS / 8;
  float top = 0.0f;
  auto soft = [&](auto i) {
    if constexpr (i < NS / 4) {
      top = fmaxf(fmaxf(i == 0 ? kNegInf : top, s.template get<4 * i>()), s.template get<4 * i + 1>());
      top = fmaxf(fmaxf(top, s.template get<4 * i + 2>()), s.template get<4 * i + 3>());
    } else if constexpr (i == NS / 4) {
      if (__any(top * p.scale2 > m + kLazy)) {
        if (!WIDE) top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float mn = fmaxf(m, top * p.scale2);
        const float a = mn == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= a;
        acc_settle();
        unroll<2 * ROWS>([&](auto t) { acc_write<t>(acc_read<t>() * a); });
        acc_settle();
      }
      top = m == kNegInf ? 0.0f : -m;
    } else if constexpr (i <= NS / 4 + NS) {
      constexpr int e = i - NS / 4 - 1;
      s.template set<e>(__builtin_amdgcn_exp2f(__builtin_fmaf(s.template get<e>(), p.scale2, top)));
      if constexpr (e > 0) l += s.template get<e - 1>();   // the one before: this one is not there at once
    } else {
      constexpr int k = i - NS / 4 - 1 - NS;
      if constexpr (k == 0) l += s.template get<NS - 1>();
      v4u u;
      unroll<4>([&](auto d) { u[(int)d] = pack2_bf16(s.template get<8 * k + 2 * d>(), s.template get<8 * k + 2 * d + 1>()); });
      pr[k] = __builtin_bit_cast(v8bf, u);
    }
  };
  auto fence = [] { __builtin_amdgcn_sched_barrier(0); };

  if constexpr (PIPE) {
    // Two tiles at once: the scores of tile k + 1 are multiplied while the probabilities of tile k are
    // made (vector instructions in the matrix instructions' shadow), then tile k's output is, while
    // tile k + 3 is asked for.  One barrier a step, put before the last kAhead products of the output,
    // whose operands are in registers by then: behind it tile k's place is free, tile k + 2 is there,
    // and the reads of its first fragments run under those products.  Tiles past the segment's end
    // are asked for too (the last token again and again), so that the counts stay the same.
    // FP8: three places.  Tile k + 2 is made of its codes under the products of tile k's output, and
    // then tile k + 4's codes are asked for, into the stage that got free, and its rotated part
    // into the place of tile k + 1, whose scores every wave has by then.
    Scores<ROWS> t;
    auto meet = [&](auto outstanding) {
      wait_vmcnt<outstanding>();
      barrier_lds();
    };
    auto next = [](int place) { return place + 1 == NT ? 0 : place + 1; };
    if (n_steps > 0) {
      if constexpr (FP8) {
        wait_vmcnt<0>();
        for (int k = 0; k < 2; ++k) {
          spread_at(raw_at + k * kRawB, tile_at + k * kTileB);
          unroll<20>([&](auto u) { spread_bit(u); });
        }
        __builtin_amdgcn_s_waitcnt(0xc07f);          // lgkmcnt(0): the codes are read before others land on them
        fetch(t_seg + 2 * STEP, tile_at + 2 * kTileB, raw_at);
        barrier_lds();
      } else {
        meet(std::integral_constant<int, 2 * NL>{});
      }
      keys_at(0);
      unroll<kAhead>([&](auto f) { key(f); });
      s.clear();
      unroll<NF>([&](auto f) {
        fence();
        score(f, s);
        if constexpr (f + kAhead < NF) key(std::integral_constant<int, f + kAhead>{});
      });
      if constexpr (FP8) {
        barrier_lds();                               // everyone has tile 0's scores: its rotated part makes room
        fetch(t_seg + 3 * STEP, tile_at, raw_at + kRawB);
      } else {
        meet(std::integral_constant<int, NL>{});
      }
      keys_at(kTileB);
      unroll<kAhead>([&](auto f) { key(f); });
    }
    int place = 0;                                   // of tile k
    for (int k = 0; k < n_steps; ++k) {
      const int tb = t_seg + k * STEP;
      values_at(place * kTileB);
      hide(k, tb, tile_at + place * kTileB);
      if (k + 1 < n_steps) {
        t.clear();
        unroll<NF>([&](auto f) {
          fence();
          score(f, t);
          if constexpr (f + kAhead < NF) key(std::integral_constant<int, f + kAhead>{});
          else value(std::integral_constant<int, f + kAhead - NF>{});
          if constexpr (f < kSoft) soft(f);
        });
      } else {
        unroll<kAhead>([&](auto f) { value(f); });
        unroll<kSoft>([&](auto i) { soft(i); });
        operands_settle();
      }
      const int two = next(next(place));             // of tile k + 2
      const int free = next(two);                    // bf16: of tile k + 3
      const uint32_t codes = raw_at + (k & 1) * kRawB;   // of tiles k + 2 and k + 4
      From f3;
      if constexpr (FP8) wait_vmcnt<NL>();           // the codes of tile k + 2, asked for two steps ago
      unroll<NV - kAhead>([&](auto f) {
        fence();
        product(f);
        value(std::integral_constant<int, f + kAhead>{});
        if constexpr (FP8) {
          if constexpr (f == 0) spread_at(codes, tile_at + two * kTileB);
          if constexpr (f < 20) spread_bit(f);
          if constexpr (f == 16) f3 = find(tb + 4 * STEP, rw);
        } else {
          if constexpr (f == 0) f3 = find(tb + 3 * STEP, rw);
          if constexpr (f >= 3 && f % 2 == 1 && f < 3 + 2 * NL) ask(f3, tile_at + free * kTileB + rw * kBlockB, 0u, std::integral_constant<int, (f - 3) / 2>{});
        }
      });
      place = next(place);
      if constexpr (FP8) barrier_lds();
      else meet(std::integral_constant<int, NL>{});
      keys_at(next(place) * kTileB);
      unroll<kAhead>([&](auto i) {
        fence();
        product(std::integral_constant<int, NV - kAhead + i>{});
        if constexpr (FP8 && i < NL) ask(f3, tile_at + place * kTileB + rw * kBlockB, codes, i);
      });
      unroll<kAhead>([&](auto f) { key(f); });
      s = t;
    }
  } else {
    for (int k = 0; k < n_steps; ++k) {
      const int tb = t_seg + k * STEP;               // first token of this wave
      uint32_t off = 0;
      if constexpr (RW > 1 && !FP8) {
        off = (k & 1) * kTileB;
        wait_vmcnt<0>();
        barrier_lds();                               // everyone's share of tile k is here, tile k - 1 is done with
        if (k + 1 < n_steps) fetch(tb + STEP, tile_at + (kTileB - off), 0u);
      } else if constexpr (RW > 1) {
        const uint32_t from = raw_at + (k & 1) * NSUB * kRawB;
        if (k + 1 < n_steps) wait_vmcnt<NSUB * NL>();
        else wait_vmcnt<0>();
        barrier_lds();                               // tile k - 1 is done with
#pragma unroll
        for (int i = 0; i < NSUB; ++i)
          unroll<5>([&](auto u) { spread_raw(rw * NSUB + i, u, from + i * kRawB, tile_at); });
        barrier_lds();                               // tile k is whole
        if (k + 2 < n_steps) fetch(tb + 2 * STEP, tile_at, from);
      } else {
        if (tb >= end_max) break;                    // the other token waves have the rest
        if constexpr (FP8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int u = 0; u < 4; ++u) spread(i, u, code_reg[4 * i + u], scale_reg[4 * i + u], tile_at);
            spread_rope(i, rope_reg[i], tile_at);
          }
          if (k + 1 < n_steps && tb + STEP < end_max) fetch_regs(tb + STEP);
        } else {
          wait_vmcnt<0>();
        }
      }
      keys_at(off);
      values_at(off);
      s.clear();
      unroll<kAhead>([&](auto f) { key(f); });
      unroll<NF>([&](auto f) {
        fence();
        score(f, s);
        if constexpr (f + kAhead < NF) key(std::integral_constant<int, f + kAhead>{});
        else value(std::integral_constant<int, f + kAhead - NF>{});
      });
      fence();
      if (hide(k, tb, tile_at + off)) unroll<kAhead>([&](auto f) { value(f); });
      unroll<kSoft>([&](auto i) { soft(i); });
      operands_settle();
      unroll<NV>([&](auto f) {
        fence();
        product(f);
        if constexpr (f + kAhead < NV) value(std::integral_constant<int, f + kAhead>{});
      });
      if constexpr (RW == 1 && !FP8)                 // its reads are over: the next tokens into the same tile
        if (k + 1 < n_steps && tb + STEP < end_max) fetch(tb + STEP, tile_at, 0u);
    }
  }
  acc_settle();

  // the row's sum over the g, then over the token waves
  {
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const int n = ln % ROWS, g = ln / ROWS;
    float* const red = reinterpret_cast<float*>(smem);   // [4 waves][m ROWS, l ROWS], then [4 waves][channels][ROWS]
    if (!WIDE) l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    float part = 1.0f;                               // this token wave's weight
    float mt = m, lt = l;
    if constexpr (TW > 1) {
      __syncthreads();
      if (g == 0) {
        red[wave * 2 * ROWS + n] = m;
        red[wave * 2 * ROWS + ROWS + n] = l;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < TW; ++k) mt = fmaxf(mt, red[(k * RW + rw) * 2 * ROWS + n]);
      const float base = mt == kNegInf ? 0.0f : mt;
      lt = 0.0f;
#pragma unroll
      for (int k = 0; k < TW; ++k) {
        const float* rk = red + (k * RW + rw) * 2 * ROWS + n;
        lt += rk[ROWS] * __builtin_amdgcn_exp2f(rk[0] - base);
      }
      part = __builtin_amdgcn_exp2f(m - base);
    }
    const int r = rw * ROWS + n;                     // row of the tile
    const bool mine = r_tile + r <= r_last;
    const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;   // (a sum that is NaN gives NaN)
    const int64_t orow = (int64_t)sq.q0 * p.H + r_tile + r;
    const int64_t slot = 2 * (int64_t)w + (step0 == 0);
    if (tw == 0 && g == 0) {
      const float lse = lt == 0.0f ? kNegInf : mt + __builtin_log2f(lt);
      if (!whole) p.part_lse[slot * M + r] = lse;
      else if (mine && p.lse) p.lse[orow] = lse * kLn2;
    }
    // group i of accumulators; a part keeps the registers' order, [RW][NG][lane][4], whole lines a store
    auto put = [&](int i, v4f v) {
      v *= inv;
      if (!whole) *reinterpret_cast<v4f*>(p.part_out + ((slot * RW + rw) * NG + i) * 256 + 4 * ln) = v;
      else if (mine) store4(p, orow * kR + GS * i + 4 * g, v);
    };
    if constexpr (TW > 1) {
      // LDS holds four waves' accumulators of NG / PASS groups at a time; token wave tw adds and
      // stores its share of them
      constexpr int PASS = ROWS / 16, PG = NG / PASS, OWN = PG / TW;
      float* ow = red + wave * PG * 4 * 64;
      unroll<PASS>([&](auto ps) {
        __syncthreads();
        unroll<PG>([&](auto i) { *reinterpret_cast<v4f*>(ow + (i * 64 + ln) * 4) = acc_read<ps * PG + i>() * part; });
        __syncthreads();
#pragma unroll 4
          for (int i = tw * OWN; i < (tw + 1) * OWN; ++i) {
            v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < TW; ++k) v += *reinterpret_cast<const v4f*>(red + (k * RW + rw) * PG * 4 * 64 + (i * 64 + ln) * 4);
            put(ps * PG + i, v);
          }
      });
    } else {
      unroll<NG>([&](auto i) { put(i, acc_read<i>()); });
    }
  }
  if (threadIdx.x == 0 && step0 == 0 && !whole) {
    // the share that finishes the tile is the first whose own end is at, or snaps to, the tile's
    const int64_t last = (plan.hi.end * plan.shares + plan.total - 1) / plan.total - 1;
    p.meta[w] = Meta{(int64_t)sq.q0 * p.H + r_tile, r_last - r_tile + 1, (int)last - w + 1};
  }
  }
  wait_vmcnt<0>();                                   // loads under way to LDS end before the workgroup does
}

// Joins the parts of split row tiles with weights 2^(lse_k - max), in the order
// of the accumulators that they were written in: a lane has one row and 4
// channels of each group, so its weights are its own.  Bound by reading the
// parts.  A workgroup finds the split tiles (a thread per share) and takes items
// of them in turn: of a tile in few parts a wave does kRun groups of one row
// wave; of one in many, the eight waves share the parts of kRunMany groups and
// meet in LDS, so that one tile in 128 parts and 128 tiles in two keep the card
// busy alike.  Measured: two tiles of 128 rows in 128 parts each (67 MB) 15 us, 4.5
// TB/s; such tiles in two to four parts (24 sequences of up to 61 new tokens, 16 heads, 70 MB) 18
// us; nothing to join 5 us.
constexpr int kGrid = 256;    // shares: the MI355X's CUs
constexpr int kJoin = 1024;   // workgroups of eight waves
constexpr int kFew = 16, kRun = 8, kRunMany = 2;
template <int ROWS>
__global__ void __launch_bounds__(512) join_kernel(AttnParams p, int RW) {
  constexpr int GS = Scores<ROWS>::TS, NG = kR / GS;
  __shared__ Meta metas[kGrid];
  __shared__ int64_t sums[8];
  __shared__ int before[kGrid + 1];
  __shared__ __attribute__((aligned(16))) float meet[8][kRunMany + 1][64][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int M = ROWS * RW;
  int64_t items = 0, all;
  if (tid < kGrid) {
    const Meta mine = p.meta[tid];
    metas[tid] = mine;
    items = mine.parts == 0 ? 0 : mine.parts <= kFew ? (RW * (NG / kRun) + 7) / 8 : RW * (NG / kRunMany);
  }
  const int64_t at = block_scan<8>(items, sums, all);
  if (tid < kGrid) before[tid] = (int)at;
  __syncthreads();
  for (int item = blockIdx.x; item < (int)all; item += gridDim.x) {
    int w = 0;                                       // the last share with before[w] <= item
#pragma unroll
    for (int s = kGrid / 2; s; s >>= 1)
      if (before[w + s] <= item) w += s;
    const Meta meta = metas[w];
    const int u = item - before[w];
    const int n = lane % ROWS, g = lane / ROWS;
    // part 0 is slot 1 of share w, part k slot 0 of share w + k
    auto slot = [&](int k) { return k == 0 ? 2 * (int64_t)w + 1 : 2 * (int64_t)(w + k); };
    auto finish = [&](int r, int i, v4f v, float inv) {
      if (r < meta.rows) store4(p, (meta.row + r) * kR + GS * i + 4 * g, v * inv);
    };
    if (meta.parts <= kFew) {
      const int unit = 8 * u + wave;
      if (unit >= RW * (NG / kRun)) continue;
      const int rw = unit / (NG / kRun), i0 = unit % (NG / kRun) * kRun, r = rw * ROWS + n;
      float top = kNegInf, sum = 0.0f;
      float lse[kFew];                               // all under way at once; the last again behind it
#pragma unroll
      for (int k = 0; k < kFew; ++k) lse[k] = p.part_lse[slot(min(k, meta.parts - 1)) * M + r];
#pragma unroll
      for (int k = 0; k < kFew; ++k) top = fmaxf(top, lse[k]);
      const float base = top == kNegInf ? 0.0f : top;
      v4f acc[kRun];
#pragma unroll
      for (int i = 0; i < kRun; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
      for (int k = 0; k < meta.parts; ++k) {
        const float x = __builtin_amdgcn_exp2f(p.part_lse[slot(k) * M + r] - base);
        const float* src = p.part_out + ((slot(k) * RW + rw) * NG + i0) * 256 + 4 * lane;
        sum += x;
#pragma unroll
        for (int i = 0; i < kRun; ++i) acc[i] += *reinterpret_cast<const v4f*>(src + i * 256) * x;
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int i = 0; i < kRun; ++i) finish(r, i0 + i, acc[i], inv);
      if (i0 == 0 && g == 0 && r < meta.rows && p.lse)
        p.lse[meta.row + r] = sum == 0.0f ? kNegInf : (top + __builtin_log2f(sum)) * kLn2;
    } else {
      const int rw = u / (NG / kRunMany), i0 = u % (NG / kRunMany) * kRunMany, r = rw * ROWS + n;
      float top = kNegInf, sum = 0.0f;
      for (int k = wave; k < meta.parts; k += 32) {
#pragma unroll
        for (int d = 0; d < 32; d += 8) top = fmaxf(top, p.part_lse[slot(min(k + d, meta.parts - 1)) * M + r]);
      }
      __syncthreads();                               // the last item's sums are used
      meet[wave][kRunMany][lane][0] = top;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, meet[k][kRunMany][lane][0]);
      const float base = top == kNegInf ? 0.0f : top;
      v4f acc[kRunMany];
#pragma unroll
      for (int i = 0; i < kRunMany; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      for (int k0 = wave; k0 < meta.parts; k0 += 32) {
#pragma unroll
        for (int d = 0; d < 32; d += 8) {            // behind the last: that one again, with weight 0
          const int k = min(k0 + d, meta.parts - 1);
          const float y = p.part_lse[slot(k) * M + r] - base, x = k0 + d < meta.parts ? __builtin_amdgcn_exp2f(y) : 0.0f;
          const float* src = p.part_out + ((slot(k) * RW + rw) * NG + i0) * 256 + 4 * lane;
          sum += x;
#pragma unroll
          for (int i = 0; i < kRunMany; ++i) acc[i] += *reinterpret_cast<const v4f*>(src + i * 256) * x;
        }
      }
#pragma unroll
      for (int i = 0; i < kRunMany; ++i) *reinterpret_cast<v4f*>(meet[wave][i][lane]) = acc[i];
      meet[wave][kRunMany][lane][1] = sum;
      __syncthreads();
      if (wave < kRunMany) {
        sum = 0.0f;
        v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v += *reinterpret_cast<const v4f*>(meet[k][wave][lane]);
          sum += meet[k][kRunMany][lane][1];
        }
        finish(r, i0 + wave, v, sum == 0.0f ? 0.0f : 1.0f / sum);
        if (i0 == 0 && wave == 0 && g == 0 && r < meta.rows && p.lse)
          p.lse[meta.row + r] = sum == 0.0f ? kNegInf : (top + __builtin_log2f(sum)) * kLn2;
      }
    }
  }
}

// The rows of a tile.  More rows read the cache fewer times and multiply at a
// better rate; fewer have less to set up, to split and to join.  The estimate is
// start + unit * (32 cached tokens' steps a share), in us, as measured with 16 to
// 128 heads, 1 to 128 sequences of 300 to 100000 tokens and 1 to 128 new ones (a
// graph of calls, bf16 / fp8; 128-row tiles: 1.75 / 1.85 us a unit when the matrix
// cores bound it).  It takes the table's width for the sequences' length, and
// when the new tokens cannot be shared out evenly half a tile a sequence as lost.
// Measured with 16 / 32 / 64 / 128 rows (us, bf16): 32 x 4096, 128 heads 98 / 84 / 69 / 79; 128
// new tokens on 8192, 128 heads 514 / 398 / 313 / 267; 32 x 4096, 16 heads 48 / 50 / 52 / 70;
// 16 new tokens each on 4 x 2000, 16 heads 34 / 37 / 41 / 52; 1 to 8 new each on 64 x up to
// 4000, 16 heads 114 / 87 / 80 / 96; fp8, 2 x 100000, 128 heads 164 / 154 / 98 / 91; fp8,
// 128 x 4096, 32 heads 118 / 119 / 132 / 170.
// A table much wider than its sequences makes short ones pay for larger tiles and the join
// (own width / 131,072 tokens): 32 x 500, 128 heads 24 / 43; 8 x 1000 27 / 39; 4 x 30 13 / 24;
// 32 x 4096 71 / 76; 16 heads the same both ways.
struct TileCost {
  int m;
  float start[2], unit[2];   // bf16, fp8
};
constexpr TileCost kTiles[] = {
    {16, {21, 22}, {0.65f, 0.8f}}, {32, {25, 26}, {1.0f, 1.3f}}, {64, {31, 31}, {1.2f, 1.4f}}, {128, {40, 42}, {1.9f, 2.2f}}};

// the largest tile that an average sequence's rows fill by half
int most_rows(int64_t T, int64_t H, int64_t B) {
  const int64_t per = (T * H + B - 1) / B;
  return per > 64 ? 128 : per > 32 ? 64 : per > 16 ? 32 : 16;
}
int tile_rows(int64_t T, int64_t H, int64_t B, int64_t len, bool fp8) {
  const int most = most_rows(T, H, B);
  int best = 16;
  double least = 1e30;
  for (const TileCost& c : kTiles) {
    if (c.m > most) break;
    const double tiles = T % B == 0 ? (double)B * ((T * H + B * c.m - 1) / (B * c.m)) : (double)T * H / c.m + 0.5 * B;
    const double us = c.start[fp8] + c.unit[fp8] * std::ceil(tiles * ((len + kTok - 1) / kTok) / kGrid);
    if (us < least) least = us, best = c.m;
  }
  return best;
}

constexpr int64_t part_bytes(int m) { return (int64_t)kGrid * 2 * m * (kR + 1) * 4; }

}  // namespace

int64_t mla_attention_workspace_bytes(int64_t T, int64_t H, int64_t B) {
  return kGrid * (int64_t)sizeof(Meta) + part_bytes(most_rows(T, H, B));
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
  // |scale|, its sign on Q; 0 is taken as 2^-126, so that masked scores stay infinite and the others vanish
  p.scale2 = std::max(fabsf(a.scale) * 1.4426950408889634f, 1.17549435e-38f);
  p.flip = a.scale < 0.0f ? 0x80008000u : 0u;
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
  p.longest = (int)std::min(a.W * a.ps, ((int64_t)1 << 31) - 4096);
  p.causal = a.causal;
  p.out_f32 = a.out_f32;
  const int m = tile_rows(a.T, a.H, a.B, a.W * a.ps, a.fp8);
  p.meta = static_cast<Meta*>(a.workspace);
  p.part_lse = reinterpret_cast<float*>(p.meta + kGrid);
  p.part_out = p.part_lse + (int64_t)kGrid * 2 * m;
#define FP8BS_ATTN(ROWS_, RW_, TW_, F8_) \
  hipLaunchKernelGGL((mla_attention_kernel<ROWS_, RW_, TW_, F8_>), dim3(kGrid), dim3(256), 0, stream, p)
  switch (m) {
    case 128:
      if (a.fp8) FP8BS_ATTN(32, 4, 1, true);
      else FP8BS_ATTN(32, 4, 1, false);
      break;
    case 64:
      if (a.fp8) FP8BS_ATTN(16, 4, 1, true);
      else FP8BS_ATTN(16, 4, 1, false);
      break;
    case 32:
      if (a.fp8) FP8BS_ATTN(16, 2, 2, true);
      else FP8BS_ATTN(16, 2, 2, false);
      break;
    default:
      if (a.fp8) FP8BS_ATTN(16, 1, 4, true);
      else FP8BS_ATTN(16, 1, 4, false);
  }
  // A table no wider than a step of the plan: tiles are one step, none is split.  (One token, 16 heads, 100
  // cached, us a call from a graph: 14.0, with the join's launch 16.0.)
  if (a.W * a.ps <= kTok * (m == 16 ? 4 : m == 32 ? 2 : 1)) return hipGetLastError();
  // no more workgroups than the split tiles can have items
  const int64_t items = std::min((int64_t)kGrid, a.T * a.H / m + a.B) * (2 * m / kRunMany);
  const dim3 join((unsigned)std::min(items, (int64_t)kJoin));
  if (m == 128) hipLaunchKernelGGL(join_kernel<32>, join, dim3(512), 0, stream, p, 4);
  else hipLaunchKernelGGL(join_kernel<16>, join, dim3(512), 0, stream, p, m / 16);
#undef FP8BS_ATTN
  return hipGetLastError();
}

}  // namespace fp8bs
