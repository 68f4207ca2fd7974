/*
 * fp8bs.h -- C ABI of the block-scaled FP8 linear library for AMD MI355X
 * (gfx950).  Every entry point takes plain device pointers, sizes and a HIP
 * stream, enqueues its kernels on that stream and returns without waiting.
 *
 * Conventions shared by all entry points
 *   - Tensors are dense, row-major and contiguous; sizes are element counts.
 *   - "e4m3" is the OCP float8 E4M3 "fn" byte format (torch.float8_e4m3fn):
 *     bias 7, no infinities, 0x7F/0xFF are NaN, largest magnitude 448.
 *   - "bf16" tensors are passed as their 16-bit patterns (torch.bfloat16).
 *   - Block size is 128 everywhere: activations carry one float32 scale per
 *     1 x 128 block along K, weights one per 128 x 128 block.  A scale is the
 *     dequantisation multiplier: real value = decode(code) * scale.
 *   - The caller owns all memory.  The library never allocates or frees
 *     device memory, creates no streams or events, and keeps no state
 *     between calls beyond a per-device cache of the compute-unit count.  It
 *     is safe to call from several host threads.
 *   - `stream` is a hipStream_t (NULL = the legacy default stream) on the
 *     current HIP device; all pointers must be device (or managed) memory of
 *     that device.
 *   - Arguments are validated on the host before any HIP call.  A non-zero
 *     status means nothing was enqueued (except FP8BS_ERR_HIP, returned when
 *     a kernel launch itself fails).  Faults inside kernels are reported
 *     asynchronously by HIP, as for any kernel.
 *   - Inputs holding NaN are outside the contract (NaN propagates; payloads
 *     are not specified).
 *
 * The operations follow the DeepSeek-V3 inference pages: "DeepSeek-V3
 * Administrator & Developer Guide" sections 8.5.1 (act_quant_kernel), 8.5.2
 * (weight_dequant_kernel), 8.5.3 (fp8_gemm_kernel), 6.3 (the FP8 path and
 * the weight scale shape), 6.4 (MoE expert loop); "DeepSeek-V3 User Guide"
 * section 7 FAQ (scale_fmt ue8m0) and section 6 (K must be a multiple of 128).
 */
#ifndef FP8BS_H
#define FP8BS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define FP8BS_OK          0
#define FP8BS_ERR_NULL    1  /* a required pointer is NULL */
#define FP8BS_ERR_SHAPE   2  /* negative size, K not a multiple of 128, size limit */
#define FP8BS_ERR_ALIGN   3  /* a pointer is not 16-byte aligned */
#define FP8BS_ERR_ENUM    4  /* unknown scale_fmt / out_dtype */
#define FP8BS_ERR_HIP     5  /* a HIP launch failed */
#define FP8BS_ERR_ALIAS   6  /* an output overlaps an input */

/* Scale formats for activation quantisation. */
#define FP8BS_SCALE_FP32  0  /* s = max(amax, 1e-4) / 448 as float32 */
#define FP8BS_SCALE_UE8M0 1  /* s rounded up to the next power of two */

/* Output element types of the GEMMs (and element types of arguments that may be either). */
#define FP8BS_OUT_BF16    0
#define FP8BS_OUT_F32     1

/* Element types of an MLA cache's latents. */
#define FP8BS_CACHE_BF16  0
#define FP8BS_CACHE_FP8   1  /* e4m3 codes with a power-of-two float32 scale per 128 */

/* Scores of the gate. */
#define FP8BS_SCORE_SIGMOID 0
#define FP8BS_SCORE_SOFTMAX 1

/* Human-readable name of a status code (static string, never NULL). */
const char* fp8bs_status_string(int status);

/* Library version as major*10000 + minor*100 + patch. */
int fp8bs_version(void);

/*
 * act_quant -- per-1x128-block activation quantisation.
 * Admin guide 8.5.1; ue8m0 per the User guide FAQ.
 *
 * For every row m and block j (columns 128j .. 128j+127):
 *   amax = max |x|,  s = RN32(max(amax, 1e-4f) / 448)   (IEEE division),
 *   ue8m0: s = smallest power of two >= s,
 *   q = e4m3(RN32(x / s))  (correctly rounded division, then round to nearest
 *   even onto the e4m3 grid, saturating at +-448).
 *
 *   x_bf16  in   bf16 [M, K]
 *   q_e4m3  out  e4m3 [M, K]          (must not overlap x)
 *   s       out  float32 [M, K/128]
 *   M >= 0 (0 = no-op), K >= 0 with K % 128 == 0 (else FP8BS_ERR_SHAPE).
 *   One launch covers at most 2^32 - 1 threads, 32 blocks per 256 threads:
 *   M * (K / 128) <= 536870880 (M * K up to about 2^36); larger shapes
 *   return FP8BS_ERR_SHAPE.
 *   All three pointers 16-byte aligned except `s` (4-byte).
 *   x must be finite: a block holding +-Inf or NaN gets an unspecified scale
 *   and unspecified codes (the rule above is not defined for it).
 */
int fp8bs_act_quant(const void* x_bf16, void* q_e4m3, float* s, int64_t M, int64_t K,
                    int scale_fmt, void* stream);

/*
 * e4m3_encode -- the float32 -> e4m3 step of act_quant and weight_quant on
 * its own (the cast to float8_e4m3fn of Admin guide 8.5.1): q[i] is x[i]
 * rounded to the nearest e4m3 value, ties to even mantissa, magnitudes
 * above 448 saturating to +-448 (464, the midpoint to the next binade,
 * rounds to 448); the sign of a zero result follows x.  Exposed so that
 * the hardware conversion can be checked against a reference over every
 * float32 input.
 *
 *   x       in   float32 [n] (16-byte aligned)
 *   q_e4m3  out  e4m3 [n] (4-byte aligned, must not overlap x)
 *   n >= 0; n <= 2^34 - 1024 (one launch), else FP8BS_ERR_SHAPE.
 *   NaN inputs are outside the contract.
 */
int fp8bs_e4m3_encode(const float* x, void* q_e4m3, int64_t n, void* stream);

/*
 * weight_quant -- 128x128-block weight quantisation with the same rule as
 * act_quant (fp32 scale format).  The pages ship weights already quantised
 * (Admin guide 6.3: one float32 scale per 128 x 128 block, shape
 * ceil(N/128) x ceil(K/128)); this entry point produces that form from a
 * bf16 weight.  A partial edge block uses the amax of its own elements.
 *
 *   w_bf16  in   bf16 [N, K]
 *   q_e4m3  out  e4m3 [N, K]
 *   s       out  float32 [ceil(N/128), ceil(K/128)]
 *   N, K >= 0, any values.
 */
int fp8bs_weight_quant(const void* w_bf16, void* q_e4m3, float* s, int64_t N, int64_t K,
                       void* stream);

/*
 * weight_dequant -- Admin guide 8.5.2:
 *   y[n, k] = bf16_RNE( RN32( decode(w[n, k]) * s[n/128, k/128] ) ).
 *
 *   w_e4m3  in   e4m3 [N, K]
 *   s       in   float32 [ceil(N/128), ceil(K/128)]
 *   y_bf16  out  bf16 [N, K]
 *   N, K >= 0, ragged edge blocks allowed.  One launch covers at most 2^32 - 1
 *   threads: N*K + 255 < 2^32 when K % 16 != 0, and ceil(N/4) * ceil(K/1024)
 *   < 2^24 workgroups when K % 16 == 0 (N*K up to about 2^36); larger shapes
 *   return FP8BS_ERR_SHAPE.
 */
int fp8bs_weight_dequant(const void* w_e4m3, const float* s, void* y_bf16, int64_t N, int64_t K,
                         void* stream);

/*
 * gemm -- block-scaled FP8 GEMM, Admin guide 8.5.3 (nn.Linear layout):
 *   C[m, n] = sum_kb ( sum_{k in block kb} a[m, k] * b[n, k] )
 *                    * a_s[m, kb] * b_s[n / 128, kb]
 * with float32 accumulation; each 128-wide K block's partial product is
 * scaled once and added to the accumulator.
 *
 *   a    in   e4m3 [M, K]              (activations, from fp8bs_act_quant)
 *   a_s  in   float32 [M, K/128]
 *   b    in   e4m3 [N, K]              (weight, out x in)
 *   b_s  in   float32 [ceil(N/128), K/128]
 *   c    out  [M, N], bf16 (RNE) or float32 per out_dtype
 *   M >= 0 (0 = no-op), N >= 0, K >= 128 with K % 128 == 0;
 *   (M + 256) * K < 2^32 and (N + 256) * K < 2^32 (32-bit operand offsets).
 *   a, b, c 16-byte aligned; a_s, b_s 4-byte aligned.
 *
 * Accuracy.  Let S[m, n] = sum_kb sum_{k in kb} |a[m,k] * b[n,k]| * a_s[m,kb]
 * * b_s[n/128,kb] (the sum of the absolute scaled products) and ref the exact
 * sum.  M <= 64 runs on bf16 matrix instructions over exactly decoded codes;
 * its float32 result carries only the float32 rounding of the accumulation,
 * within about (K/128 + 16) * 2^-24 * S of ref.  M > 64 runs on the FP8 matrix instruction
 * (K = 128 per instruction), whose internal sum of a block's 128 products is
 * not exact in float32: measured on gfx950 its error per block reaches about
 * 1.4e-5 of the block's sum of |products| on normally distributed codes and
 * 2^-13.6 of it with 1% of activations scaled by 50.  The float32 result
 * then satisfies |err| <= 1e-2 * |ref| + 1e-3 + 2^-11 * S.  Where products
 * cancel (|ref| much smaller than S) the first two terms alone can be missed:
 * with 1% x50 activation outliers about 1 output in 10^4 did (211 of 1.57 M
 * at 1024 x 1536 x 7168); on N(0,1) activations none were seen.  A bf16
 * output adds its own rounding, 2^-9 * |ref|.
 */
int fp8bs_gemm(const void* a, const float* a_s, const void* b, const float* b_s, void* c,
               int64_t M, int64_t N, int64_t K, int out_dtype, void* stream);

/*
 * moe_gemm -- grouped block-scaled FP8 GEMM over E experts in one launch,
 * the per-expert products of the MoE loop (Admin guide 6.4), each computed as
 * in fp8bs_gemm.  Rows [offsets[e], offsets[e+1]) of `a` (grouped by expert)
 * are multiplied by expert e's weight:
 *   C[r, n] = sum_kb (sum_k a[r, k] * b[e, n, k]) * a_s[r, kb] * b_s[e, n/128, kb].
 *
 *   a        in   e4m3 [R, K]
 *   a_s      in   float32 [R, K/128]
 *   b        in   e4m3 [E, N, K]
 *   b_s      in   float32 [E, ceil(N/128), K/128]
 *   offsets  in   DEVICE int32 [E+1]: offsets[0] = 0, non-decreasing,
 *                 offsets[E] = R (precondition, not checked on the host so
 *                 that no device->host copy is needed; the kernel clamps
 *                 every range to [0, R] so a violation cannot write outside c)
 *   c        out  [R, N] bf16 or float32; rows not covered by any expert are
 *                 left untouched
 *   R, E >= 0 (either 0 = no-op), N >= 0, K >= 128 with K % 128 == 0;
 *   (R + 256) * K < 2^32 and (N + 256) * K < 2^32.
 * One launch on `stream`: experts with more than 64 rows run on the 256 x 256
 * tiles of fp8bs_gemm, the others on 64 x 256 tiles that stream the weight
 * once, the two kinds of tiles sharing the grid.  The grid is sized on the
 * host from R and E alone (each workgroup finds its tile from the device
 * offsets, so no device-to-host copy is needed); experts with no rows cost
 * nothing.  Accuracy as fp8bs_gemm for M > 64 (both tile kinds use the FP8
 * matrix instruction).
 */
int fp8bs_moe_gemm(const void* a, const float* a_s, const void* b, const float* b_s,
                   const int32_t* offsets, void* c, int64_t R, int64_t E, int64_t N, int64_t K,
                   int out_dtype, void* stream);

/*
 * gemm_ue8m0 -- fp8bs_gemm for operands whose scales are all powers of two
 * (act_quant with FP8BS_SCALE_UE8M0 and fp8bs_weight_quant_ue8m0), the ue8m0
 * variant of the pages (User guide FAQ; Admin guide 8.5.1).  The result is the
 * same sum; the kernel passes each scale's exponent to the MFMA
 * (v_mfma_scale_f32_16x16x128_f8f6f4, E8M0 scales) instead of folding the
 * scales in with VALU instructions.  Arguments as fp8bs_gemm.
 * PRECONDITION (not checked on the host: the scales live on the device):
 * every a_s and b_s value is 2^k with -126 <= k <= 127; only the exponent
 * field is read, so other values give wrong results, not faults.
 * Accuracy as fp8bs_gemm: M > 64 uses the same FP8 matrix instruction
 * (scaled form) and has the same 2^-11 * S term beyond
 * 1e-2 * |ref| + 1e-3; M <= 64 runs fp8bs_gemm's bf16 decode kernel.
 */
int fp8bs_gemm_ue8m0(const void* a, const float* a_s, const void* b, const float* b_s, void* c,
                     int64_t M, int64_t N, int64_t K, int out_dtype, void* stream);

/*
 * weight_quant_ue8m0 -- fp8bs_weight_quant with each block scale rounded up
 * to a power of two (act_quant's ue8m0 rule on 128 x 128 blocks); a harness
 * option: the pages round only activation scales.  Arguments as
 * fp8bs_weight_quant.
 */
int fp8bs_weight_quant_ue8m0(const void* w_bf16, void* q_e4m3, float* s, int64_t N, int64_t K,
                             void* stream);

/*
 * w8a16_gemm -- the BF16 path of the linear (Admin guide 6.3, gemm_impl
 * "bf16"): C = x . weight_dequant(w, w_s)^T with the weight dequantised as
 * fp8bs_weight_dequant does (bf16(RN32(decode(q) * s))) but never stored:
 * the kernel dequantises in registers and multiplies with bf16 MFMA,
 * accumulating in float32.
 *
 *   x_bf16   in   bf16 [M, K]
 *   w_e4m3   in   e4m3 [N, K] (nn.Linear out x in)
 *   w_s      in   float32 [ceil(N/128), K/128]
 *   c        out  [M, N] bf16 or float32 (out_dtype)
 *   M, N >= 0 (either 0 = no-op), K >= 128 with K % 128 == 0;
 *   (M + 256) * 2K < 2^32 and (N + 256) * K < 2^32.
 * x, w and c 16-byte aligned, w_s 4-byte aligned; c must not overlap an input.
 */
int fp8bs_w8a16_gemm(const void* x_bf16, const void* w_e4m3, const float* w_s, void* c, int64_t M,
                     int64_t N, int64_t K, int out_dtype, void* stream);

/*
 * MoE dispatch and combine -- the steps around fp8bs_moe_gemm in the expert
 * loop of the Admin guide (6.4; the annotated forward pass in 8.4): hit
 * counts of the routed expert ids, each expert's (token, slot) pairs in token
 * order, the expert run on those tokens' rows, and the expert outputs scaled
 * by the routing weight of their (token, slot) and summed per token.
 *
 * moe_route_workspace_size -- bytes of device workspace fp8bs_moe_route
 * needs for T tokens, topk slots and E experts (4 * ceil(T*topk/512) * E;
 * 0 when T*topk == 0).  Returns -1 for sizes fp8bs_moe_route rejects.
 */
int64_t fp8bs_moe_route_workspace_size(int64_t T, int64_t topk, int64_t E);

/*
 * moe_route -- stable counting sort of the routed expert ids by expert.
 *
 *   indices    in   DEVICE int32 [T, topk]: the expert of each (token, slot)
 *   offsets    out  DEVICE int32 [E+1]: expert e owns rows [offsets[e],
 *                   offsets[e+1]); offsets[E] = R, the number of pairs whose
 *                   id lies in [0, E)
 *   row_token  out  DEVICE int32 [T*topk]: the token of each row r < R, rows
 *                   of one expert in (token, slot) order (the order the
 *                   pages' per-expert index lookup yields); entries >= R
 *                   untouched
 *   row_of     out  DEVICE int32 [T, topk]: the row of each (token, slot), or
 *                   -1 when its id is outside [0, E) (such a pair is not
 *                   routed and takes no row)
 *   workspace  tmp  DEVICE, >= fp8bs_moe_route_workspace_size bytes, 4-byte
 *                   aligned; its contents are scratch (nothing needs clearing)
 *   T >= 0, 1 <= topk, 1 <= E, T*topk < 2^31.  Two kernel launches (four
 *   when ceil(T*topk/512) * E > 65536 or E > 2048); the result does not
 *   depend on timing (its only atomics are on-chip adds and ORs, whose order
 *   does not change it).
 */
int fp8bs_moe_route(const int32_t* indices, int64_t T, int64_t topk, int64_t E, int32_t* offsets,
                    int32_t* row_token, int32_t* row_of, void* workspace,
                    int64_t workspace_bytes, void* stream);

/*
 * moe_route_noalloc -- fp8bs_moe_route with no workspace argument, for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation).  The count table
 * lives in a 1 MiB device array inside the library (one per GPU, held until
 * the process ends); the call allocates nothing.  Limit:
 * fp8bs_moe_route_workspace_size(T, topk, E) <= 1048576 bytes, i.e.
 * ceil(T*topk/512) * E <= 262144 (e.g. 4096 tokens x top-8 with up to 4096
 * experts), else FP8BS_ERR_SHAPE.  Every call on one GPU uses the same
 * table: calls that overlap in time on one GPU (on different streams, or
 * from several host threads without ordering) race and give wrong results.
 * Other arguments, results and errors as fp8bs_moe_route.
 */
int fp8bs_moe_route_noalloc(const int32_t* indices, int64_t T, int64_t topk, int64_t E,
                            int32_t* offsets, int32_t* row_token, int32_t* row_of, void* stream);

/*
 * moe_quant_scatter -- the expert inputs: act_quant (as fp8bs_act_quant) of
 * every token row of x, written to each row its (token, slot) pairs were
 * routed to.  Quantisation is row local, so row r holds act_quant of
 * x[row_token[r]].
 *
 *   x        in   bf16 [T, K], K % 128 == 0
 *   row_of   in   DEVICE int32 [T, topk] (from fp8bs_moe_route); entries
 *                 outside [0, R) are skipped
 *   q        out  e4m3 [R, K]; s out float32 [R, K/128]; rows no pair maps
 *                 to are left untouched
 *   scale_fmt     FP8BS_SCALE_FP32 or FP8BS_SCALE_UE8M0
 * Alignment as fp8bs_act_quant; row_of 4-byte aligned.  If row_of maps two
 * pairs to one row, that row receives one of the two (identical for a
 * token's own duplicates).  Launch limit as fp8bs_act_quant with M = T:
 * T * (K / 128) <= 536870880, else FP8BS_ERR_SHAPE.
 */
int fp8bs_moe_quant_scatter(const void* x_bf16, const int32_t* row_of, void* q_e4m3, float* s,
                            int64_t T, int64_t topk, int64_t R, int64_t K, int scale_fmt,
                            void* stream);

/*
 * moe_combine -- y[t, n] = sum_k w[t, k] * out[row_of[t, k], n], summed in
 * float32 in slot order (the pages accumulate y in place, expert by expert;
 * here a token's at most topk terms are summed once and rounded once).
 *
 *   out      in   bf16 [R, N]: expert outputs in routed-row order
 *   w        in   float32 [T, topk]: routing weights
 *   row_of   in   DEVICE int32 [T, topk]; pairs outside [0, R) contribute 0
 *   y        out  [T, N] bf16 or float32 (out_dtype); overwritten, not
 *                 accumulated into
 * out and y 16-byte aligned, w and row_of 4-byte aligned; N >= 0, T >= 0,
 * topk >= 1, R >= 0.
 */
int fp8bs_moe_combine(const void* out_bf16, const float* w, const int32_t* row_of, void* y,
                      int64_t T, int64_t topk, int64_t R, int64_t N, int out_dtype, void* stream);

/*
 * MLA absorb with an FP8 wkv_b -- the two products of the absorb attention
 * (Admin guide 8.3, steps 5 and 7) that use the up-projection wkv_b
 * [H*(dn+dv), R] viewed per head as [H, dn+dv, R].  With an FP8 wkv_b the
 * pages dequantise the whole weight (weight_dequant, 8.5.2) on every forward
 * step and then run the einsums; here the kernels dequantise in registers
 * with the same rounding (bf16(RN32(decode(q) * s))) and multiply with bf16
 * MFMA, accumulating in float32; the bf16 weight is never stored.
 *
 * mla_absorb_key -- q_nope carried into the latent space by the key rows:
 *   out[t, h, c] = sum_{d < dn} q[t, h, d] * Wd[h*(dn+dv) + d, c]
 * mla_absorb_value -- the attention-weighted latent turned into values by
 * the value rows:
 *   out[t, h, d] = sum_{c < R} x[t, h, c] * Wd[h*(dn+dv) + dn + d, c]
 *
 *   q_bf16 / x_bf16  in   bf16, element (t, h, i) at [t*ld_t + h*ld_h + i]
 *                         for i < dn (key) or i < R (value); ld_t, ld_h >= 0
 *                         and multiples of 8 (so the q_nope slice of a
 *                         [T, H, dn + rope] q can be passed in place)
 *   wkv_b            in   e4m3 [H*(dn+dv), R]
 *   wkv_b_s          in   float32 [H*(dn+dv)/128, R/128]
 *   out              out  contiguous [T, H, R] (key) or [T, H, dv] (value),
 *                         bf16 or float32 (out_dtype)
 *   dn, dv, R positive multiples of 128 (the pages' configurations all use
 *   128, 128, 512); key side: dn is 128 or 256; value side: R <= 512.
 *   T, H >= 0 (either 0 = no-op); the weight, the output and the input's
 *   extent below 2^31 elements.
 * Input, wkv_b and out 16-byte aligned, wkv_b_s 4-byte aligned; out must not
 * overlap an input (FP8BS_ERR_ALIAS).
 */
int fp8bs_mla_absorb_key(const void* q_bf16, int64_t ld_t, int64_t ld_h, const void* wkv_b,
                         const float* wkv_b_s, void* out, int64_t T, int64_t H, int64_t dn,
                         int64_t dv, int64_t R, int out_dtype, void* stream);
int fp8bs_mla_absorb_value(const void* x_bf16, int64_t ld_t, int64_t ld_h, const void* wkv_b,
                           const float* wkv_b_s, void* out, int64_t T, int64_t H, int64_t dn,
                           int64_t dv, int64_t R, int out_dtype, void* stream);

/*
 * The paged MLA cache -- what the absorb attention keeps of a token (Admin
 * guide 8.3: kv_cache and pe_cache), in pages, and the attention between
 * fp8bs_mla_absorb_key and fp8bs_mla_absorb_value.
 *
 * Shared by the entry points below:
 *   latent     DEVICE [P, ps, 512]: the normalised latents, bf16
 *              (FP8BS_CACHE_BF16) or e4m3 codes (FP8BS_CACHE_FP8)
 *   rope       DEVICE bf16 [P, ps, 64]: the rotated part of the shared key
 *   lat_scale  DEVICE float32 [P, ps, 4] with FP8BS_CACHE_FP8 (NULL otherwise):
 *              the multipliers of 128 codes each, powers of two in 2^-100 ..
 *              2^100, so that code * scale is exact in bf16
 *   table      DEVICE int32 [B, W]: the pages of sequence b in order; token j
 *              lies in page table[b][j / ps] at j % ps.  Entries behind the
 *              sequence's last page are not read.
 *   lens       DEVICE int32 [B]: tokens of each sequence, 0 .. W * ps, those
 *              of this call included
 *   cu_q       DEVICE int32 [B + 1]: sequence b's new tokens are rows cu_q[b]
 *              .. cu_q[b+1] - 1; cu_q[0] = 0, non-decreasing, cu_q[B] <= T.
 *              A sequence may have none.  Its new tokens are its last: with
 *              n_b of them, the i-th has position lens[b] - n_b + i.
 *   R = 512 and dr = 64 (the pages' configurations all use these).
 *   1 <= ps <= 4096, P >= 1, 1 <= W <= 2^30, P * ps < 2^31, a sequence of at most
 *   2^31 - 4096 tokens.
 * Values of table, lens and cu_q lie on the device and are preconditions, not
 * checked on the host; the kernels clamp lens to [0, W * ps] (the attention also to
 * 2^31 - 4096) and cu_q to [0, T],
 * never write outside the cache, and read no page outside [0, P), so a wrong
 * value gives wrong results for its sequence, not faults (a cu_q that decreases:
 * for the batch).
 * latent, rope and lat_scale do not overlap (the entry points that write them check).
 * Byte and bf16 pointers and lat_scale are 16-byte aligned, the other float32 and
 * the int32 ones 4-byte, a bf16 norm_w 2-byte.
 */

/*
 * mla_cache_write -- the new tokens into the cache, and their queries rotated:
 *   c = kv[t, 0:512] / sqrt(mean(kv[t, 0:512]^2) + eps) * norm_w
 *   latent <- bf16(c), or per 128: s = the power of two of act_quant's
 *             FP8BS_SCALE_UE8M0 rule on c, code = e4m3(c / s)
 *   rope   <- bf16(rotate(kv[t, 512:576])),  q_out[t, h] = bf16(rotate(q[t, h]))
 * where rotate turns each pair (2i, 2i + 1) by the angle whose cosine and sine
 * are rope_cs[position][i] (the interleaved pairs of the pages' complex
 * product).  The sum of squares, the norm and the products are float32,
 * rounded once.
 *
 *   q_rope   in   bf16, element (t, h, i) at [t*ldq_t + h*ldq_h + i], i < 64:
 *                 the rope slice of the query; ldq_t, ldq_h >= 0, multiples of 8
 *   kv       in   bf16, element (t, i) at [t*ld_kv + i], i < 576; multiple of 8
 *   norm_w   in   [512] float32 (norm_w_f32 != 0) or bf16
 *   eps           0 .. 3e38
 *   rope_cs  in   float32 [n_pos, 32, 2]: (cos, sin)
 *   q_out    out  bf16 [T, H, 64]
 *   0 <= T < 2^24 (0 = no-op), H >= 0 (0 = no queries), 0 <= B <= 2^30 (0 =
 *   no-op), n_pos >= 0.
 * A token at a position outside [0, n_pos) is skipped: neither its cache row
 * nor its q_out is written.  A token whose page lies outside [0, P) has its
 * q_out written only.  Rows t >= cu_q[B] are left as they were.  Two tokens
 * of one call must not share a cache row (a page that two sequences share is
 * made one's own by fp8bs_cache_update first).
 */
int fp8bs_mla_cache_write(const void* q_rope, int64_t ldq_t, int64_t ldq_h, const void* kv,
                          int64_t ld_kv, const void* norm_w, int norm_w_f32, float eps,
                          const float* rope_cs, int64_t n_pos, void* q_out, void* latent,
                          float* lat_scale, void* rope, int cache_fmt, const int32_t* table,
                          const int32_t* cu_q, const int32_t* lens, int64_t T, int64_t H, int64_t B,
                          int64_t W, int64_t P, int64_t ps, int64_t R, int64_t dr, void* stream);

/*
 * mla_attention -- the new tokens' attention over the cache:
 *   s[t, h, j] = scale * (q_lat[t, h] . c_j + q_rope[t, h] . k_j),
 *   out[t, h]  = sum_j softmax_j(s[t, h, :]) c_j
 *   lse[t, h]  = log sum_j exp(s[t, h, j])
 * over the tokens j of t's sequence: j <= position(t) when causal, else all
 * lens[b].  c_j is the cached latent (code * scale for an FP8 cache), k_j its
 * rope part.  A row that sees no token (a sequence of length 0, a position
 * below 0) gives out = 0 and lse = -inf, and so does one whose scores are all
 * -inf.  Rows t >= cu_q[B] are left as they were.
 *
 *   q_lat    in   bf16, element (t, h, i) at [t*ldq_t + h*ldq_h + i], i < 512
 *                 (fp8bs_mla_absorb_key's output)
 *   q_rope   in   bf16, the same with ldr_t, ldr_h, i < 64
 *                 (fp8bs_mla_cache_write's q_out); strides >= 0, multiples of 8
 *   scale         |scale| <= 2.3e38; one below 2^-126 / log2(e) is taken as that
 *                 (0: the scores vanish, as long as the products are below 2^100)
 *   out      out  [T, H, 512] bf16 or float32 (out_dtype)
 *   lse      out  float32 [T, H], or NULL
 *   workspace     DEVICE, >= fp8bs_mla_attention_workspace_size(T, H, B) bytes,
 *                 16-byte aligned; scratch (nothing needs clearing), not to be
 *                 shared by calls that may run at the same time.  At most 135 MB,
 *                 which more than 64 rows (tokens x heads) a sequence take
 *   T, B >= 0 (either 0 = no-op), H >= 1, T * H < 2^31, B <= 8192.
 * Products are of bf16 values (an FP8 cache's are exact in bf16) and summed in
 * float32; the probabilities are rounded to bf16 for the second product (so a
 * float32 out, the sums as they are, still differs by up to 2^-8 of the weighted
 * |c_j|), the softmax's maximum and sum are float32.  The work is laid out for
 * sequences as long as the table is wide, so a table much wider than they are
 * costs time (32 x 500 tokens, 128 heads: 24 us, in a table for 131,072 43).
 * A token that a row does not see has no part in it, whatever it holds
 * (infinities and NaN too); a row that sees a NaN is NaN, and so is one with a
 * score of +inf (lse too).  A score of -inf weighs its token with 0, which leaves
 * NaN in the channels where its latent is infinite and nowhere else.  The result
 * does not depend on timing.
 */
int64_t fp8bs_mla_attention_workspace_size(int64_t T, int64_t H, int64_t B);
int fp8bs_mla_attention(const void* q_lat, int64_t ldq_t, int64_t ldq_h, const void* q_rope,
                        int64_t ldr_t, int64_t ldr_h, const void* latent, const float* lat_scale,
                        const void* rope, int cache_fmt, const int32_t* table, const int32_t* cu_q,
                        const int32_t* lens, float scale, int causal, void* out, int out_dtype,
                        float* lse, int64_t T, int64_t H, int64_t B, int64_t W, int64_t P,
                        int64_t ps, int64_t R, int64_t dr, void* workspace, int64_t workspace_bytes,
                        void* stream);

/*
 * cache_update -- the pages of the next step: N new rows from B old ones.
 * New row i continues old row parent[i] (any other value: an empty row) and
 * is to hold new_lens[i] tokens: it keeps the first min(lens[parent],
 * new_lens) tokens in the parent's pages and, if it is longer, gets pages for
 * the rest.  So a row continued twice is forked, one that nobody continues is
 * freed, one given fewer tokens is truncated, one given more grows.
 *
 * Pages are given out in row order, lowest index first, from those that no old
 * row uses (a page freed by this call is free for the next).  Rows share what
 * they keep; a row that will write into a kept page (it grows and that page is
 * not full) shares it only as the page's keeper, the lowest such row among
 * those that keep the most of the page's tokens; any other gets a copy: a page
 * of its own with the kept tokens.  A row for which too few pages are left
 * is not grown: lens_out[i] is then what it keeps (the pages that it asked for
 * count as given out for the rows after it).
 *
 *   table, lens  in   old rows [B, W], [B]
 *   parent, new_lens  in   DEVICE int32 [N]; new_lens is clamped to [0, W * ps]
 *   table_out    out  DEVICE int32 [N, W], -1 behind each row's last page
 *   lens_out     out  DEVICE int32 [N]
 *   latent, lat_scale, rope   in/out: only pages that no old row uses are
 *                     written, and only a copy's kept tokens
 *   workspace    DEVICE, >= fp8bs_cache_update_workspace_size(B, N, W, P) bytes
 *                (0 for small tables: NULL then),
 *                16-byte aligned, scratch; not shared by concurrent calls
 *   B >= 0, 0 <= N < 2^18 (N = 0: no-op), B + N < 2^24.
 * The result depends on the inputs alone, and a repeated call gives it again.
 *
 * cache_compact -- the n pages that the rows use moved to pages 0 .. n - 1:
 * pages in use at n and above go to the unused ones below n, both in
 * ascending order; table_out is the table with the new indices (-1 behind
 * each row's last page and for entries outside [0, P)), count = n.
 *   table_out    out  DEVICE int32 [B, W];  count  out  DEVICE int32 [1]
 *   workspace    >= fp8bs_cache_compact_workspace_size(B, W, P) bytes, as above
 *   0 <= B < 2^24
 */
int64_t fp8bs_cache_update_workspace_size(int64_t B, int64_t N, int64_t W, int64_t P);
int fp8bs_cache_update(void* latent, float* lat_scale, void* rope, int cache_fmt,
                       const int32_t* table, const int32_t* lens, const int32_t* parent,
                       const int32_t* new_lens, int32_t* table_out, int32_t* lens_out, int64_t B,
                       int64_t N, int64_t W, int64_t P, int64_t ps, int64_t R, int64_t dr,
                       void* workspace, int64_t workspace_bytes, void* stream);
int64_t fp8bs_cache_compact_workspace_size(int64_t B, int64_t W, int64_t P);
int fp8bs_cache_compact(void* latent, float* lat_scale, void* rope, int cache_fmt,
                        const int32_t* table, const int32_t* lens, int32_t* table_out,
                        int32_t* count, int64_t B, int64_t W, int64_t P, int64_t ps, int64_t R,
                        int64_t dr, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * What stands between the FP8 products of a block with experts (Admin guide
 * 1.1 and 8.4): the norm in front of them, the gate that makes the ids and
 * weights of fp8bs_moe_route and fp8bs_moe_combine, its balance loss, the
 * activation between an expert's two products; and their gradients, those of
 * fp8bs_moe_combine among them.  (The gradient of fp8bs_moe_quant_scatter is
 * fp8bs_moe_combine with weights of 1.)
 *
 * rmsnorm -- with the residual's addition and FP8 output:
 *   t = x + res (x without a residual),  c = t / sqrt(mean(t^2) + eps) * norm_w
 *   res_out = t rounded to its type,  y = bf16(c)
 *   per 128 columns: s by act_quant's rule on c, q = e4m3(c / s), the quotient
 *   within two roundings (a product with 1 / s)
 * All in float32 from the inputs on, each output rounded once: the norm is
 * that of the unrounded sum, the codes are those of the unrounded norm.  A row
 * whose squares sum to infinity in float32 gives zeros (NaN where it is infinite
 * itself), as does one of zeros; with eps = 0 the latter is NaN.
 * Codes where c is not finite, for swiglu's too: a block with an infinity has an
 * infinite scale, the codes of its finite values are 0 and those of its infinities
 * NaN; a NaN has the code of a NaN, and the scale is that of the block's other
 * values.
 *
 *   x        in   bf16, element (m, k) at [m*ld_x + k]; ld_x >= 0, a multiple of 8
 *   res      in   [M, K] bf16 or float32 (res_dtype, FP8BS_OUT_*), or NULL
 *   res_out  out  [M, K] of res's type; may be res itself.  NULL with res NULL
 *   norm_w   in   [K] float32 (norm_w_f32 != 0) or bf16
 *   eps           0 .. 3e38
 *   y        out  bf16 [M, K], or NULL
 *   q, s     out  e4m3 [M, K] and float32 [M, K/128], or both NULL; y or q is there
 *   scale_fmt     FP8BS_SCALE_FP32 or FP8BS_SCALE_UE8M0
 *   0 <= M <= 4194303 (67108860 for K <= 512), K % 128 == 0, 0 <= K <= 32768 (M
 *   or K 0: no-op).
 * All pointers 16-byte aligned but s (4).
 *
 * rmsnorm_bwd -- of y by the norm's input h (x, or res_out) and by norm_w:
 *   g = dy * norm_w, r = 1 / sqrt(mean(h^2) + eps)
 *   dx = r * (g - h * r^2 * mean(g * h)) + dres,   dw = sum over rows of dy * h * r
 * dx is the gradient of x and of res alike; dres is what reaches res_out from
 * elsewhere.  The codes' rounding is passed straight through.  A row whose
 * squares sum to infinity, which forward gives zeros, has dx = dres (as long as
 * g * h sums to a number) and adds nothing to dw.
 *   dy       in   bf16 [M, K]
 *   h        in   bf16 or float32 (h_dtype), element (m, k) at [m*ld_h + k]
 *   dres     in   [M, K] of h's type, or NULL; may be dx itself
 *   dx       out  [M, K] of h's type
 *   dw       out  float32 [K] (M = 0: zeros), or NULL
 *   workspace     DEVICE, >= fp8bs_rmsnorm_bwd_workspace_size(M, K) bytes (not
 *                 needed without dw; 0 for few rows), 16-byte aligned, scratch,
 *                 not shared by calls that may run at the same time
 * The sums are float32 in a fixed order: the result does not depend on timing.
 */
int fp8bs_rmsnorm(const void* x_bf16, int64_t ld_x, const void* res, void* res_out, int res_dtype,
                  const void* norm_w, int norm_w_f32, float eps, void* y_bf16, void* q_e4m3, float* s,
                  int scale_fmt, int64_t M, int64_t K, void* stream);
int64_t fp8bs_rmsnorm_bwd_workspace_size(int64_t M, int64_t K);
int fp8bs_rmsnorm_bwd(const void* dy_bf16, const void* h, int64_t ld_h, int h_dtype, const void* norm_w,
                      int norm_w_f32, float eps, const void* dres, void* dx, float* dw, int64_t M, int64_t K,
                      void* workspace, int64_t workspace_bytes, void* stream);

/*
 * moe_gate -- the experts and routing weights of every token:
 *   score = sigmoid(logit), or softmax over the token's logits
 *   key = float32(score) + bias; the logit itself where there is no bias (the
 *         scores have its order)
 *   groups > 1: the experts lie in `groups` runs of E / groups; a group counts
 *         as the sum of its two largest keys (without a bias: its largest);
 *         only the topk_groups groups that count most are looked at
 *   indices = the topk largest keys' experts, the largest first
 *   weights = score / (sum of the chosen scores, if normalize) * route_scale
 * Ties go to the lowest index, among groups too.  An expert whose logit is -inf
 * or NaN is masked: its score is 0, a softmax leaves it out, and it is never
 * chosen; nor is one whose key is -inf or NaN.  Slots for which no expert is left
 * hold index -1, which fp8bs_moe_route does not route, and weight 0.  Logits of
 * +inf share a softmax's weight.  With a bias the scores are computed in 64
 * bits and rounded once, so that the choice does not turn on the last bit of
 * an exponential; all else is float32.
 *
 *   logits   in   float32 or bf16 (logits_dtype), element (t, e) at [t*ld + e], ld >= 0
 *   bias     in   float32 [E], or NULL
 *   indices  out  int32 [T, topk];  weights  out  float32 [T, topk]
 *   score         FP8BS_SCORE_SIGMOID or FP8BS_SCORE_SOFTMAX
 *   0 <= T < 2^24 (0 = no-op), 1 <= E <= 1024, 1 <= topk <= min(E, 64),
 *   1 <= topk_groups <= groups <= 64, E % groups == 0; route_scale finite.
 *
 * moe_balance -- per-expert counts and the balance loss of each sequence s,
 * tokens cu_seq[s] .. cu_seq[s+1] - 1, n of them:
 *   counts[s, e] = how often its tokens' indices name e
 *   probs[s, e]  = mean over its tokens of score_e / (sum of the token's scores)
 *   loss[s]      = E / (topk * n) * sum_e counts[s, e] * probs[s, e]
 * (1 where all experts are used alike).  A sequence without tokens gives zeros;
 * a token whose experts are all masked (as above) adds no shares; indices outside
 * [0, E) are not counted.
 *   indices  in   int32 [T, topk] (from fp8bs_moe_gate)
 *   cu_seq   in   DEVICE int32 [S + 1], non-decreasing, or NULL: one sequence
 *                 of all T tokens, S = 1.  The values are a precondition, not
 *                 checked on the host: wrong ones give wrong results, not faults
 *   counts   out  int32 [S, E];  probs  out  float32 [S, E];  loss  out  float32 [S]
 *   workspace     DEVICE, >= fp8bs_moe_balance_workspace_size(T, S, E) bytes (0:
 *                 NULL), 16-byte aligned, scratch, not shared by concurrent calls
 *   0 <= S < 2^22 (0 = no-op); T = 0 gives zeros.
 *
 * moe_gate_bwd -- the gradient by the logits of both: of the weights, given
 * d_weights, and of the losses, given d_loss (the counts and the choice of
 * experts are constants):
 *   d_weights in  float32 [T, topk], or NULL (no part); needs indices
 *   d_loss    in  float32 [S], or NULL (no part); needs counts of fp8bs_moe_balance
 *   d_logits  out float32 or bf16 (out_dtype) [T, E], 16-byte aligned; 0 for masked
 *             experts.  Tokens outside all sequences get d_weights' part alone
 *   score, normalize, route_scale  as given to fp8bs_moe_gate
 * An index that a token names twice counts twice; one outside [0, E) is left
 * out.  Sums of no scores (all underflowed or masked) give 0.
 * Results do not depend on timing.  Pointers are aligned to their elements.
 */
int fp8bs_moe_gate(const void* logits, int64_t ld, int logits_dtype, const float* bias, int64_t T, int64_t E,
                   int64_t topk, int64_t groups, int64_t topk_groups, int score, int normalize, float route_scale,
                   int32_t* indices, float* weights, void* stream);
int64_t fp8bs_moe_balance_workspace_size(int64_t T, int64_t S, int64_t E);
int fp8bs_moe_balance(const void* logits, int64_t ld, int logits_dtype, const int32_t* indices, const int32_t* cu_seq,
                      int64_t T, int64_t S, int64_t E, int64_t topk, int score, int32_t* counts, float* probs,
                      float* loss, void* workspace, int64_t workspace_bytes, void* stream);
int fp8bs_moe_gate_bwd(const void* logits, int64_t ld, int logits_dtype, const int32_t* indices,
                       const float* d_weights, int score, int normalize, float route_scale, const int32_t* cu_seq,
                       const int32_t* counts, const float* d_loss, int64_t T, int64_t S, int64_t E, int64_t topk,
                       void* d_logits, int out_dtype, void* stream);

/*
 * swiglu -- the activation between an expert's two products:
 *   a = g * sigmoid(g) * u   (float32),  y = bf16(a),
 *       (to float32's accuracy also where sigmoid(g) is below its range, to g = -174)
 *   per 128 columns: s by act_quant's rule on a, q = e4m3(a / s) as rmsnorm's
 *   gate, up in   bf16, element (m, n) at [m*ld + n]: two tensors, or the halves
 *                 of one; ld_g, ld_u >= 0, multiples of 8
 *   n_rows   in   DEVICE int32 [1], or NULL: rows from *n_rows (clamped to [0, M])
 *                 on are neither read nor written (offsets + E of fp8bs_moe_route)
 *   y        out  bf16 [M, N], or NULL;  q, s  out  e4m3 [M, N] and float32
 *                 [M, N/128], or both NULL; y or q is there
 *   M, N >= 0 (either 0 = no-op), N % 128 == 0, M * N < about 2^37 (one launch).
 *
 * swiglu_bwd --
 *   du = dy * g * sig,  dg = dy * u * sig * (1 + g * (1 - sig)),  sig = sigmoid(g)
 *   dy       in   bf16 [M, N]
 *   dgate, dup  out  bf16, strided as gate and up are (ld >= N for more than one
 *                 row); they may be columns of the same rows, but share no element
 * All pointers 16-byte aligned but s and n_rows (4).
 *
 * moe_combine_bwd -- the gradient of fp8bs_moe_combine:
 *   d_out[row_of[t, k]] = bf16(w[t, k] * dy[t]),  d_w[t, k] = <dy[t], out[row_of[t, k]]>
 *   dy       in   bf16 or float32 (dy_dtype) [T, N]
 *   out      in   bf16 [R, N];  w, row_of  in  float32, int32 [T, topk]
 *   d_out    out  bf16 [R, N]; rows that no pair maps to are left untouched
 *   d_w      out  float32 [T, topk]; 0 for pairs outside [0, R)
 *   0 <= T < 2^23, topk >= 1, T * topk < 2^31, R, N >= 0.
 * If row_of maps two pairs to one row, each element of that row of d_out
 * receives either's.
 * dy, out and d_out 16-byte aligned, the others 4-byte.
 */
int fp8bs_swiglu(const void* gate_bf16, int64_t ld_g, const void* up_bf16, int64_t ld_u, const int32_t* n_rows,
                 void* y_bf16, void* q_e4m3, float* s, int scale_fmt, int64_t M, int64_t N, void* stream);
int fp8bs_swiglu_bwd(const void* dy_bf16, const void* gate_bf16, int64_t ld_g, const void* up_bf16, int64_t ld_u,
                     const int32_t* n_rows, void* dgate_bf16, int64_t ld_dg, void* dup_bf16, int64_t ld_du,
                     int64_t M, int64_t N, void* stream);
int fp8bs_moe_combine_bwd(const void* dy, int dy_dtype, const void* out_bf16, const float* w, const int32_t* row_of,
                          void* d_out_bf16, float* d_w, int64_t T, int64_t topk, int64_t R, int64_t N, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BS_H */
