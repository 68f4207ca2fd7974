// mla_cache.hip -- the paged MLA latent cache for gfx950: new tokens into it,
// and its pages from one step to the next.
//
// A cache of P pages of ps tokens is three dense arrays, as the pages'
// kv_cache and pe_cache are two ("DeepSeek-V3 Administrator & Developer Guide"
// 8.3): latent [P, ps, 512] (bf16, or e4m3 codes), rope bf16 [P, ps, 64], and
// for codes scale float32 [P, ps, 4], one power of two per 128 latents.  A
// power-of-two scale makes code * scale exact in bf16, so the attention's
// matrix operands are the cached values themselves.
#include <algorithm>
#include <cstdint>

#include "device_common.h"
#include "launch.h"

namespace fp8bs {

namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr int kR = 512, kD = 64;

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// ---------------------------------------------------------------------------
// cache write: one workgroup per token.  Wave 0 normalises the latent (eight
// channels a lane), rotates the shared key and stores both; the other waves
// rotate the heads' query parts, 16 bytes a lane.  All lanes of a wave share
// the token, so its sequence is found 64 boundaries at a time.  HBM-bound:
// 4096 tokens of 128 heads into an FP8 cache (57 MB) in 13.1 us, 4.4 TB/s of the
// 4.9 that a copy reaches; 32 tokens 5.2 us, a launch and four dependent reads
// (boundaries, length, page, data).  The norm and the rotation are float32
// throughout; what is stored is rounded once, to bf16 or e4m3, as the cache's type says.
// ---------------------------------------------------------------------------
struct WriteParams {
  const uint16_t* q;       // [T, H, 64] by ldq_t, ldq_h
  const uint16_t* kv;      // [T, 576] by ld_kv
  const void* w;           // [512]
  const float* cs;         // [n_pos, 32, 2]
  uint16_t* q_out;         // [T, H, 64]
  uint8_t* latent;
  float* scale;
  uint16_t* rope;
  const int32_t *table, *cu_q, *lens;
  int64_t ldq_t, ldq_h, ld_kv, n_pos;
  float eps;
  int T, H, B, W, P, ps;
  int w_f32;
};

// b = the number of boundaries cu_q[1 .. B] at or below t, found by the whole wave
__device__ __forceinline__ int find_seq(const int32_t* cu_q, int B, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = B;                                // the answer is in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 63) / 64;
    const int at = lo + (lane + 1) * step;          // boundary `at` bounds `at` sequences
    const bool le = at <= lo + n && cu_q[min(at, B)] <= t;
    lo += __popcll(__ballot(le)) * step;
    n = min(step - 1, max(B - lo, 0));
  }
  return lo;
}

// pairs (2i, 2i + 1) of four packed dwords turned by (cos, sin) i
__device__ __forceinline__ v4u rotate8(v4u x, const float* cs) {
  v4u r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = bf16_lo(x[i]), b = bf16_hi(x[i]), c = cs[2 * i], d = cs[2 * i + 1];
    r[i] = pack2_bf16(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, d)), __fadd_rn(__fmul_rn(a, d), __fmul_rn(b, c)));
  }
  return r;
}

template <bool FP8>
__global__ void __launch_bounds__(256) mla_cache_write_kernel(WriteParams p) {
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 63;
  const int b = find_seq(p.cu_q, p.B, t);
  if (b >= p.B || t < p.cu_q[b]) return;             // a row behind the last sequence
  if (t >= p.cu_q[b + 1]) return;                    // boundaries that decrease: below, pos < len holds for the others
  const int64_t len = min((int64_t)max(p.lens[b], 0), (int64_t)p.W * p.ps);
  const int64_t pos = len - min(p.cu_q[b + 1], p.T) + t;
  if (pos < 0 || pos >= p.n_pos) return;
  const float* csrow = p.cs + pos * kD;

  if (threadIdx.x >= 64) {
    const int c = threadIdx.x & 7;                   // pairs 4c .. 4c + 3 of a head
    float cs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = csrow[8 * c + i];
    for (int h = (threadIdx.x - 64) >> 3; h < p.H; h += 24) {
      const v4u x = *reinterpret_cast<const v4u*>(p.q + t * p.ldq_t + h * p.ldq_h + 8 * c);
      *reinterpret_cast<v4u*>(p.q_out + ((int64_t)t * p.H + h) * kD + 8 * c) = rotate8(x, cs);
    }
    return;
  }

  const int64_t pj = pos / p.ps;
  const int pg = p.table[(int64_t)b * p.W + pj];
  if (pg < 0 || pg >= p.P) return;
  const int64_t row = (int64_t)pg * p.ps + (pos - pj * p.ps);
  const uint16_t* kv = p.kv + t * p.ld_kv;

  const v4u xw = *reinterpret_cast<const v4u*>(kv + 8 * lane);
  float x[8], ss = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(xw[i]);
    x[2 * i + 1] = bf16_hi(xw[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(x[i], x[i], ss);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) ss += __shfl_xor(ss, d);
  const float inv = 1.0f / sqrtf(ss * (1.0f / kR) + p.eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float w = p.w_f32 ? static_cast<const float*>(p.w)[8 * lane + i]
                            : bits_f32((uint32_t) static_cast<const uint16_t*>(p.w)[8 * lane + i] << 16);
    x[i] = __fmul_rn(__fmul_rn(x[i], inv), w);
  }
  if (FP8) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, f32_bits(x[i]) & 0x7FFFFFFFu);
    const float s = block_scale<true>(bits_f32(row16_max_u32(top)));
    const float r = 1.0f / s;                        // exact: s is a power of two
    const v2u q = {pack4_e4m3(x[0] * r, x[1] * r, x[2] * r, x[3] * r),
                   pack4_e4m3(x[4] * r, x[5] * r, x[6] * r, x[7] * r)};
    *reinterpret_cast<v2u*>(p.latent + row * kR + 8 * lane) = q;
    if ((lane & 15) == 0) p.scale[row * (kR / 128) + (lane >> 4)] = s;
  } else {
    const v4u v = {pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]), pack2_bf16(x[4], x[5]), pack2_bf16(x[6], x[7])};
    *reinterpret_cast<v4u*>(p.latent + row * (2 * kR) + 16 * lane) = v;
  }
  if (lane < 8) {
    float cs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = csrow[8 * lane + i];
    *reinterpret_cast<v4u*>(p.rope + row * kD + 8 * lane) =
        rotate8(*reinterpret_cast<const v4u*>(kv + kR + 8 * lane), cs);
  }
}

// ---------------------------------------------------------------------------
// cache update and compact.  Both derive the pages in use from (table, lens)
// alone, write a new table beside the old one, and copy page data only from
// pages that the old table uses to pages that it does not, so no copy reads
// what another writes and a call repeated on the same inputs gives the same.
//   mark   used bits from the old table; for update, each new row bids for the
//          pages it keeps (a maximum, so order does not matter)
//   plan   prefix sums over the rows and over the bitmap
//   apply  the new table, and the copies
// Small ones are one launch: every workgroup marks and plans for itself, in LDS,
// and applies its share, so nothing passes between workgroups and nothing waits.
// What does not fit, or makes that reading the longer part (below, at the
// launchers), goes through four launches and the workspace.
// ---------------------------------------------------------------------------
struct CacheArrays {
  uint8_t* p[3];
  int row_bytes[3];       // bytes per token, 0 = no such array
};

struct PageParams {
  CacheArrays c;
  const int32_t *table, *lens;        // old [B, W], [B]
  const int32_t *parent, *new_lens;   // update: [N]
  int32_t *table_out, *lens_out;      // update: [N, W], [N]; compact: [B, W]
  int32_t* count;                     // compact: pages in use
  // workspace
  uint32_t* used;                     // ceil(P / 32) words
  int32_t* key;                       // update: [P]
  int32_t* list;                      // update: free pages; compact: holes, then movers
  int32_t* rowinfo;                   // update: [N, 4]: first new slot, new pages, their rank, copy
  int32_t* before;                    // compact: used pages before each word
  int32_t* total;                     // compact: pages in use, pages to move
  int B, W, P, ps, N, words;
};

constexpr int kRowBits = 18;
constexpr int kRowTop = (1 << kRowBits) - 1;

__device__ __forceinline__ int pages_of(int n, int ps) { return (int)(((int64_t)n + ps - 1) / ps); }

// A new row: where it comes from and what it keeps
struct Row {
  int parent, keep, kept, want;
  bool grows;             // it writes into its last kept page
};
__device__ __forceinline__ Row load_row(const PageParams& p, int i) {
  Row r;
  const int64_t most = (int64_t)p.W * p.ps;
  r.parent = p.parent[i];
  if (r.parent < 0 || r.parent >= p.B) r.parent = -1;
  r.want = (int)min((int64_t)max(p.new_lens[i], 0), most);
  const int have = r.parent < 0 ? 0 : (int)min((int64_t)max(p.lens[r.parent], 0), most);
  r.keep = min(have, r.want);
  r.kept = pages_of(r.keep, p.ps);
  r.grows = r.want > r.keep && r.keep % p.ps != 0;
  return r;
}
// the row's bid for its slot-th kept page: the most kept tokens, then the lowest row that grows into it
__device__ __forceinline__ int bid(const PageParams& p, const Row& r, int i, int slot) {
  const int tok = min(r.keep - slot * p.ps, p.ps);
  return (tok << kRowBits) | (r.grows && slot == r.kept - 1 ? kRowTop - i : 0);
}

__global__ void __launch_bounds__(256) page_clear_kernel(PageParams p) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < p.words) p.used[i] = 0;
  if (p.key && i < p.P) p.key[i] = 0;
}

__global__ void __launch_bounds__(256) page_mark_kernel(PageParams p) {
  const int r = blockIdx.x;
  if (r < p.B) {
    const int n = pages_of((int)min((int64_t)max(p.lens[r], 0), (int64_t)p.W * p.ps), p.ps);
    for (int j = threadIdx.x; j < n; j += 256) {
      const int g = p.table[(int64_t)r * p.W + j];
      if (g >= 0 && g < p.P) atomicOr(&p.used[g >> 5], 1u << (g & 31));
    }
    return;
  }
  const int i = r - p.B;
  const Row row = load_row(p, i);
  for (int j = threadIdx.x; j < row.kept; j += 256) {
    const int g = p.table[(int64_t)row.parent * p.W + j];
    if (g >= 0 && g < p.P) atomicMax(&p.key[g], bid(p, row, i, j));
  }
}

// exclusive prefix sum over the workgroup's 1024 threads; total gets the sum
template <typename I>
__device__ __forceinline__ I block_scan(I v, I* sums, I& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const I x = wave_scan(v);
  __syncthreads();
  if (lane == 63) sums[wave] = x;
  __syncthreads();
  I base = 0;
  total = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    if (k < wave) base += sums[k];
    total += sums[k];
  }
  return base + x - v;
}

__global__ void __launch_bounds__(1024) page_plan_update_kernel(PageParams p) {
  __shared__ int sums[16];
  __shared__ int64_t long_sums[16];                  // 1024 rows may ask for more than 2^31 pages
  int n_free = 0;
  for (int w0 = 0; w0 < p.words; w0 += 1024) {
    const int w = w0 + threadIdx.x;
    uint32_t bits = 0;
    if (w < p.words) {
      bits = ~p.used[w];
      if (w == p.P / 32) bits &= (1u << (p.P & 31)) - 1;
    }
    int total, at = n_free + block_scan((int)__popc(bits), sums, total);
    for (; bits; bits &= bits - 1) p.list[at++] = 32 * w + __ffs(bits) - 1;
    n_free += total;
  }
  int64_t base = 0;
  for (int i0 = 0; i0 < p.N; i0 += 1024) {
    const int i = i0 + threadIdx.x;
    Row row{};
    int need = 0;
    bool copy = false;
    if (i < p.N) {
      row = load_row(p, i);
      if (row.want > row.keep) {
        if (row.grows) {
          const int g = p.table[(int64_t)row.parent * p.W + row.kept - 1];
          copy = g >= 0 && g < p.P && p.key[g] != bid(p, row, i, row.kept - 1);
        }
        need = pages_of(row.want, p.ps) - row.kept + copy;
      }
    }
    int64_t total;
    const int64_t at = base + block_scan((int64_t)need, long_sums, total);
    base += total;
    if (i < p.N) {
      const bool ok = need == 0 || at + need <= n_free;
      int32_t* info = p.rowinfo + 4 * (int64_t)i;
      info[0] = row.kept - (ok && copy);
      info[1] = ok ? need : 0;
      info[2] = (int)min(at, (int64_t)p.P);
      info[3] = ok && copy ? row.keep % p.ps : 0;
      p.lens_out[i] = ok ? row.want : row.keep;
    }
  }
}

// a share of the bytes of `tokens` tokens of page `from` to page `to`: the arrays' 16-byte pieces in
// one row, eight loads a thread under way before their stores
template <int THREADS>
__device__ __forceinline__ void copy_tokens(const PageParams& p, int from, int to, int tokens, int part, int parts) {
  int64_t src[3], dst[3];                            // byte addresses, less those of the pieces before
  int end[3], n = 0;
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    const int64_t page = (int64_t)p.ps * p.c.row_bytes[a];
    src[a] = (int64_t)(uintptr_t)p.c.p[a] + from * page - 16 * (int64_t)n;
    dst[a] = (int64_t)(uintptr_t)p.c.p[a] + to * page - 16 * (int64_t)n;
    n += (int)((int64_t)tokens * p.c.row_bytes[a] / 16);
    end[a] = n;
  }
  constexpr int U = 8;
  for (int i0 = part * THREADS + threadIdx.x; i0 < n; i0 += parts * THREADS * U) {
    v4u v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * parts * THREADS;
      if (i < n) v[u] = *reinterpret_cast<const v4u*>((i < end[0] ? src[0] : i < end[1] ? src[1] : src[2]) + 16 * (int64_t)i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * parts * THREADS;
      if (i < n) *reinterpret_cast<v4u*>((i < end[0] ? dst[0] : i < end[1] ? dst[1] : dst[2]) + 16 * (int64_t)i) = v[u];
    }
  }
}

// the k-th (from 0) set bit of a word
__device__ __forceinline__ int nth_bit(uint32_t v, int k) {
  for (; k; --k) v &= v - 1;
  return __ffs(v) - 1;
}
// Index of the k-th set (SET) or clear bit of a bitmap with the number of set bits before each word
template <bool SET>
__device__ __forceinline__ int select(const uint32_t* used, const int* before, int words, int k) {
  int w = 0;                                         // the last word with at most k such bits before it
  for (int n = words; n > 1;) {
    const int half = n / 2;
    if ((SET ? before[w + half] : 32 * (w + half) - before[w + half]) <= k) w += half;
    n -= half;
  }
  return 32 * w + nth_bit(SET ? used[w] : ~used[w], k - (SET ? before[w] : 32 * w - before[w]));
}

// f(row, slot, page) for every page of n rows, pages_in(row) of them at row_at(row): a wave takes every
// sixteenth row, 64 slots at a time, four rows' loads under way
template <typename Pages, typename At, typename F>
__device__ __forceinline__ void for_pages(const PageParams& p, int n, const Pages& pages_in, const At& row_at, const F& f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int j = lane; j < p.W + lane; j += 64)
    for (int r0 = wave; r0 < n; r0 += 64) {
      int g[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = r0 + 16 * u;
        g[u] = r < n && j < pages_in(r) ? row_at(r)[j] : -1;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (g[u] >= 0 && g[u] < p.P) f(r0 + 16 * u, j, g[u]);
    }
}

// used bits of the old table's entries, in LDS; ends with a barrier
__device__ __forceinline__ void mark_used(const PageParams& p, uint32_t* used) {
  for_pages(
      p, p.B,
      [&](int r) { return pages_of((int)min((int64_t)max(p.lens[r], 0), (int64_t)p.W * p.ps), p.ps); },
      [&](int r) { return p.table + (int64_t)r * p.W; },
      [&](int, int, int g) { atomicOr(&used[g >> 5], 1u << (g & 31)); });
  __syncthreads();
}
// the number of set bits before each word; returns all of them.  Ends with a barrier.
__device__ __forceinline__ int count_before(const uint32_t* used, int* before, int words, int* sums) {
  int all = 0;
  for (int w0 = 0; w0 < words; w0 += 1024) {
    const int w = w0 + threadIdx.x;
    int total;
    const int at = all + block_scan(w < words ? (int)__popc(used[w]) : 0, sums, total);
    if (w < words) before[w] = at;
    all += total;
  }
  __syncthreads();
  return all;
}

// what one launch takes: update's pages, rows and table entries, compact's pages and entries
constexpr int kSmallPages = 1 << 14, kSmallRows = 512, kSmallEntries = 45 << 10;
constexpr int kCompactPages = 1 << 17, kCompactEntries = 1 << 14;

__global__ void __launch_bounds__(1024) update_small_kernel(PageParams p, int parts) {
  __shared__ int key[kSmallPages];
  __shared__ uint32_t used[kSmallPages / 32];
  __shared__ int before[kSmallPages / 32];
  __shared__ Row rows[kSmallRows];
  __shared__ int info[kSmallRows][4];                // first new slot, new pages, their rank, tokens to copy
  __shared__ int sums[16];
  const int tid = threadIdx.x;
  for (int i = tid; i < p.P; i += 1024) key[i] = 0;
  for (int i = tid; i < p.words; i += 1024) used[i] = 0;
  for (int i = tid; i < p.N; i += 1024) rows[i] = load_row(p, i);
  __syncthreads();
  for_pages(
      p, p.N, [&](int i) { return rows[i].kept; }, [&](int i) { return p.table + (int64_t)max(rows[i].parent, 0) * p.W; },
      [&](int i, int j, int g) { atomicMax(&key[g], bid(p, rows[i], i, j)); });
  mark_used(p, used);
  const int n_free = p.P - count_before(used, before, p.words, sums);
  int64_t base = 0;
  for (int i0 = 0; i0 < p.N; i0 += 1024) {
    const int i = i0 + tid;
    Row row{};
    int need = 0;
    bool copy = false;
    if (i < p.N) {
      row = rows[i];
      if (row.want > row.keep) {
        if (row.grows) {
          const int g = p.table[(int64_t)row.parent * p.W + row.kept - 1];
          copy = g >= 0 && g < p.P && key[g] != bid(p, row, i, row.kept - 1);
        }
        need = pages_of(row.want, p.ps) - row.kept + copy;
      }
    }
    int total;
    const int64_t at = base + block_scan(need, sums, total);
    base += total;
    if (i < p.N) {
      const bool ok = need == 0 || at + need <= n_free;
      info[i][0] = row.kept - (ok && copy);
      info[i][1] = ok ? need : 0;
      info[i][2] = (int)min(at, (int64_t)p.P);
      info[i][3] = ok && copy ? row.keep % p.ps : 0;
      if (blockIdx.x == 0) p.lens_out[i] = ok ? row.want : row.keep;
    }
  }
  __syncthreads();
  for (int item = blockIdx.x; item < p.N * parts; item += gridDim.x) {
    const int i = item / parts, part = item - i * parts;
    const int first = info[i][0], need = info[i][1], rank = info[i][2], cut = info[i][3];
    const int64_t old = (int64_t)max(rows[i].parent, 0) * p.W;
    if (part == 0)
      for (int j = tid; j < p.W; j += 1024) {
        int g = -1;
        if (j >= first && j < first + need) g = select<false>(used, before, p.words, rank + j - first);
        else if (j < rows[i].kept) g = p.table[old + j];
        p.table_out[(int64_t)i * p.W + j] = g;
      }
    if (cut) copy_tokens<1024>(p, p.table[old + first], select<false>(used, before, p.words, rank), cut, part, parts);
  }
}

__global__ void __launch_bounds__(1024) compact_small_kernel(PageParams p) {
  __shared__ uint32_t used[kCompactPages / 32];
  __shared__ int before[kCompactPages / 32];
  __shared__ int sums[16];
  const int tid = threadIdx.x;
  for (int i = tid; i < p.words; i += 1024) used[i] = 0;
  __syncthreads();
  mark_used(p, used);
  const int live = count_before(used, before, p.words, sums);
  auto rank = [&](int g) { return before[g >> 5] + __popc(used[g >> 5] & ((1u << (g & 31)) - 1)); };
  const int kept = live < p.P ? rank(live) : live;   // of the pages in use, those below `live`
  if (blockIdx.x == 0 && tid == 0) *p.count = live;
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int n = pages_of((int)min((int64_t)max(p.lens[b], 0), (int64_t)p.W * p.ps), p.ps);
    for (int j = tid; j < p.W; j += 1024) {
      int g = j < n ? p.table[(int64_t)b * p.W + j] : -1;
      if (g < 0 || g >= p.P) g = -1;
      else if (g >= live) g = select<false>(used, before, p.words, rank(g) - kept);
      p.table_out[(int64_t)b * p.W + j] = g;
    }
  }
  // the rows' blocks have had their work: copies go from the other end
  for (int k = gridDim.x - 1 - blockIdx.x; k < live - kept; k += gridDim.x)
    copy_tokens<1024>(p, select<true>(used, before, p.words, kept + k), select<false>(used, before, p.words, k), p.ps, 0, 1);
}

__global__ void __launch_bounds__(256) page_apply_update_kernel(PageParams p) {
  const int i = blockIdx.x;
  const int32_t* info = p.rowinfo + 4 * (int64_t)i;
  const int first = info[0], need = info[1], rank = info[2], cut = info[3];
  const int par = p.parent[i];
  const int64_t old = (int64_t)(par < 0 || par >= p.B ? 0 : par) * p.W;
  const int kept = pages_of(min(p.lens_out[i], load_row(p, i).keep), p.ps);
  if (blockIdx.y == 0)
    for (int j = threadIdx.x; j < p.W; j += 256) {
      int g = -1;
      if (j >= first && j < first + need) g = p.list[rank + j - first];
      else if (j < kept) g = p.table[old + j];
      p.table_out[(int64_t)i * p.W + j] = g;
    }
  if (cut) copy_tokens<256>(p, p.table[old + first], p.list[rank], cut, blockIdx.y, gridDim.y);
}

__global__ void __launch_bounds__(1024) page_plan_compact_kernel(PageParams p) {
  __shared__ int sums[16];
  int live = 0;
  for (int w0 = 0; w0 < p.words; w0 += 1024) {
    const int w = w0 + threadIdx.x;
    const int c = w < p.words ? __popc(p.used[w]) : 0;
    int total;
    const int at = live + block_scan(c, sums, total);
    if (w < p.words) p.before[w] = at;
    live += total;
  }
  __syncthreads();
  // holes below `live` and used pages from there on, both ascending; as many of one as of the other
  int32_t* holes = p.list;
  int32_t* movers = p.list + p.P;
  const int split = live;
  const int kept = split < p.P ? p.before[split >> 5] + __popc(p.used[split >> 5] & ((1u << (split & 31)) - 1)) : live;
  for (int w = threadIdx.x; w < p.words; w += 1024) {
    const uint32_t u = p.used[w];
    const int lo = 32 * w, k = clampi(split - lo, 0, 32);
    const uint32_t below = k == 32 ? 0xFFFFFFFFu : (1u << k) - 1;
    int at = lo - p.before[w];                       // free pages before this word
    for (uint32_t f = ~u & below; f; f &= f - 1) holes[at++] = lo + __ffs(f) - 1;
    at = p.before[w] + __popc(u & below) - kept;
    for (uint32_t f = u & ~below; f; f &= f - 1) movers[at++] = lo + __ffs(f) - 1;
  }
  if (threadIdx.x == 0) {
    p.total[0] = kept;
    p.total[1] = live - kept;
    *p.count = live;
  }
}

// the first B blocks write a table row each; all blocks share the copies
__global__ void __launch_bounds__(256) page_apply_compact_kernel(PageParams p) {
  const int kept = p.total[0], moves = p.total[1];
  const int live = *p.count;
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int n = pages_of((int)min((int64_t)max(p.lens[b], 0), (int64_t)p.W * p.ps), p.ps);
    for (int j = threadIdx.x; j < p.W; j += 256) {
      int g = j < n ? p.table[(int64_t)b * p.W + j] : -1;
      if (g < 0 || g >= p.P) g = -1;
      else if (g >= live) {
        const int at = p.before[g >> 5] + __popc(p.used[g >> 5] & ((1u << (g & 31)) - 1)) - kept;
        g = p.list[at];
      }
      p.table_out[(int64_t)b * p.W + j] = g;
    }
  }
  for (int k = blockIdx.x; k < moves; k += gridDim.x) copy_tokens<256>(p, p.list[p.P + k], p.list[k], p.ps, 0, 1);
}

// One launch when a workgroup's LDS holds the pages' keys and the rows (86 KB) and its own
// reading of the tables takes no longer than three launches more.  us a call from a graph, one
// launch / four, fp8, by table entries (B + N) W: 16 rows of 2000 tokens 8.1 / 12.8; 64 rows to 256 with
// 10,560 13.8 / 15.9, 20,480 14.1 / 17.2, 30,400 18.0 / 18.5, 40,640 18.5 / 19.0, 50,560 21.8 / 19.0, 60,480
// 22.8 / 19.1; 128 rows with 32,512 17.1 / 16.8; 16 to 512 with 33,792 21.1 / 23.4, 50,160 27.0 / 23.7.
// Calls that are not in a graph pay the host's time for each launch (22 for four): with 50,560 20.6 / 22.3.
// The line is drawn between those on which the graph's calls lose and the others.
bool update_is_small(int64_t B, int64_t N, int64_t W, int64_t P) {
  return P <= kSmallPages && N <= kSmallRows && (B + N) * W <= kSmallEntries;
}
// The same for compact (one / four): 300 pages 6.3 / 12.7, 8192 pages with 60 rows (298 MB moved)
// 70.2 / 74.4, 12,800 entries 86.5 / 86.6, 50,800 entries 299 / 279.
bool compact_is_small(int64_t B, int64_t W, int64_t P) { return P <= kCompactPages && B * W <= kCompactEntries; }

int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

PageParams page_params(const PageTask& a) {
  PageParams p{};
  const void* ptr[3] = {a.latent, a.rope, a.scale};
  const int bytes[3] = {a.fp8 ? kR : 2 * kR, 2 * kD, a.fp8 ? kR / 128 * 4 : 0};
  for (int i = 0; i < 3; ++i) {
    p.c.p[i] = static_cast<uint8_t*>(const_cast<void*>(ptr[i]));
    p.c.row_bytes[i] = bytes[i];
  }
  p.table = a.table;
  p.lens = a.lens;
  p.parent = a.parent;
  p.new_lens = a.new_lens;
  p.table_out = a.table_out;
  p.lens_out = a.lens_out;
  p.count = a.count;
  p.B = (int)a.B;
  p.W = (int)a.W;
  p.P = (int)a.P;
  p.ps = (int)a.ps;
  p.N = (int)a.N;
  p.words = (int)((a.P + 31) / 32);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  auto take = [&](int64_t n) {
    int32_t* at = reinterpret_cast<int32_t*>(ws);
    ws += up16(4 * n);
    return at;
  };
  p.used = reinterpret_cast<uint32_t*>(take(p.words));
  if (a.parent) {
    p.key = take(a.P);
    p.list = take(a.P);
    p.rowinfo = take(4 * a.N);
  } else {
    p.before = take(p.words);
    p.list = take(2 * a.P);
    p.total = take(2);
  }
  return p;
}

}  // namespace

int64_t cache_update_workspace_bytes(int64_t B, int64_t N, int64_t W, int64_t P) {
  if (update_is_small(B, N, W, P)) return 0;
  return up16(4 * ((P + 31) / 32)) + 2 * up16(4 * P) + up16(16 * N);
}
int64_t cache_compact_workspace_bytes(int64_t B, int64_t W, int64_t P) {
  if (compact_is_small(B, W, P)) return 0;
  return 2 * up16(4 * ((P + 31) / 32)) + up16(8 * P) + 16;
}

hipError_t launch_mla_cache_write(const MlaCacheWrite& a, hipStream_t stream) {
  WriteParams p{};
  p.q = static_cast<const uint16_t*>(a.q);
  p.kv = static_cast<const uint16_t*>(a.kv);
  p.w = a.w;
  p.cs = a.cs;
  p.q_out = static_cast<uint16_t*>(a.q_out);
  p.latent = static_cast<uint8_t*>(a.latent);
  p.scale = a.scale;
  p.rope = static_cast<uint16_t*>(a.rope);
  p.table = a.table;
  p.cu_q = a.cu_q;
  p.lens = a.lens;
  p.ldq_t = a.ldq_t;
  p.ldq_h = a.ldq_h;
  p.ld_kv = a.ld_kv;
  p.n_pos = a.n_pos;
  p.eps = a.eps;
  p.T = (int)a.T;
  p.H = (int)a.H;
  p.B = (int)a.B;
  p.W = (int)a.W;
  p.P = (int)a.P;
  p.ps = (int)a.ps;
  p.w_f32 = a.w_f32;
  if (a.fp8) hipLaunchKernelGGL(mla_cache_write_kernel<true>, dim3(p.T), dim3(256), 0, stream, p);
  else hipLaunchKernelGGL(mla_cache_write_kernel<false>, dim3(p.T), dim3(256), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_cache_update(const PageTask& a, hipStream_t stream) {
  const PageParams p = page_params(a);
  if (update_is_small(a.B, a.N, a.W, a.P)) {
    const int parts = std::max(1, 256 / p.N);        // workgroups a row's copy is cut over
    hipLaunchKernelGGL(update_small_kernel, dim3(std::min(256, p.N * parts)), dim3(1024), 0, stream, p, parts);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(page_clear_kernel, dim3((p.P + 255) / 256), dim3(256), 0, stream, p);
  hipLaunchKernelGGL(page_mark_kernel, dim3(p.B + p.N), dim3(256), 0, stream, p);
  hipLaunchKernelGGL(page_plan_update_kernel, dim3(1), dim3(1024), 0, stream, p);
  hipLaunchKernelGGL(page_apply_update_kernel, dim3(p.N, 4), dim3(256), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_cache_compact(const PageTask& a, hipStream_t stream) {
  const PageParams p = page_params(a);
  if (compact_is_small(a.B, a.W, a.P)) {
    const int grid = std::min(512, std::max(1, std::max(p.P / 2, p.B)));
    hipLaunchKernelGGL(compact_small_kernel, dim3(grid), dim3(1024), 0, stream, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(page_clear_kernel, dim3((p.words + 255) / 256), dim3(256), 0, stream, p);
  if (p.B) hipLaunchKernelGGL(page_mark_kernel, dim3(p.B), dim3(256), 0, stream, p);
  hipLaunchKernelGGL(page_plan_compact_kernel, dim3(1), dim3(1024), 0, stream, p);
  const int grid = std::max(std::min(p.P / 2, 2048), std::min(p.B, 2048));
  hipLaunchKernelGGL(page_apply_compact_kernel, dim3(std::max(grid, 1)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace fp8bs
