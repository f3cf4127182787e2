/*
 * moe_operators.h -- the operators around a cache of experts, for callers that
 * hold their tensors themselves: the router, 4-bit quantisation, products grouped
 * by expert, and the weighted sum of the experts' rows.  Same library as
 * moe_cache.h (libmoecache.so), same status codes, moe_dtype values and
 * moe_last_error().
 *
 * One layer, router to output, is
 *   moe_route (logits -> ids, gates, pairs in expert order)
 *   moe_quantize_fp4 (rows gathered by expert) or the bf16 rows as they are
 *   moe_grouped_matmul / _fp4 with act = 1 (gate/up product and SwiGLU)
 *   moe_grouped_matmul / _fp4 (down product)
 *   moe_combine (sum over each token's experts)
 *
 * Conventions for every call:
 *  - Every pointer is device memory of the current device, owned by the caller.
 *    Work is enqueued on `stream` (a cudaStream_t passed as void*, NULL = legacy
 *    default stream); the host never waits and nothing is allocated, so every
 *    call can be captured in a CUDA graph.  The caller orders `stream` behind what
 *    makes the inputs, and keeps them and the outputs until the work is done.
 *  - Matrices are row-major and contiguous.  int32 / fp32 arrays are 4-byte
 *    aligned, matrices 16-byte aligned where a row of them is a multiple of 16
 *    bytes (MOE_EINVAL otherwise, before anything is enqueued).
 *  - T = 0 is allowed everywhere and enqueues what it must (empty offsets).
 *  - Results do not depend on the order in which blocks run: the same inputs give
 *    the same bits.
 *  - Every wait inside a kernel is bounded.  One that runs out sets a flag that
 *    moe_operators_check() reports; the outputs of that call are undefined.
 *
 * Expert order.  A pair p = t * k + j is token t's j-th expert.  Grouped row i
 * holds pair order[i]; the rows of expert e are offsets[e] .. offsets[e + 1] - 1,
 * pairs ascending; place[p] is the row of pair p.  tiles[e] counts the 128-row
 * tiles of the experts before e, each expert's rows starting a new tile.  moe_route and
 * moe_group_pairs make them from any ids.  The other calls do not check that what they hold
 * is a grouping; whatever it is, they read and write inside the arrays of these sizes only.
 *
 * 4-bit matrices (MOE_NVFP4, MOE_MXFP4).  codes [rows, K/2]: two e2m1 codes a
 * byte, the even element low.  scales: tiles of 128 rows x 4 blocks, 512 bytes,
 * [row tiles, ceil(K / (4 * block)), 512]: the scale of tile row r and block b of
 * the group is byte (r % 32) * 16 + (r / 32) * 4 + b.  That is the order in which
 * the tensor cores take block scales, so a product moves whole tiles.  Blocks and
 * rows past the matrix's end pad their tile; blocks pad with scale 0.  A stack of
 * G matrices of N rows starts every matrix on a new row tile; rows grouped by
 * expert start every expert on a new one (tile tiles[e]).  NVFP4: block 16, e4m3
 * scale, and one fp32 scale g per matrix; MXFP4: block 32, e8m0 scale.  Products and
 * dequantisation multiply MXFP4 values by a g too if one is given; quantising takes none.
 */
#ifndef MOE_OPERATORS_H
#define MOE_OPERATORS_H

#include "moe_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Row tiles that hold P grouped rows of at most E experts: what `scales` is sized for. */
int64_t moe_grouped_tiles(int64_t P, int32_t E);

/* Bytes of scratch for moe_route / moe_group_pairs with grouping of T tokens, k experts each, out of E. */
int64_t moe_group_workspace(int32_t T, int32_t k, int32_t E);

/*
 * The router.  logits [T, E] in logits_dtype (MOE_F32 or MOE_BF16) -> topk_ids [T, k]
 * int32, topk_w [T, k] fp32, best expert first, equal scores to the lower index.
 *   scoring 0  softmax: experts by logit; w = exp(l - max) over the sum of the k
 *              picked (renormalize = 1) or of all E (0).  bias must be NULL, n_group 1.
 *   scoring 1  sigmoid: s = 1 / (1 + exp(-l)); experts by s + bias (bias [E] fp32 or
 *              NULL); w = s, over the sum of the k picked when renormalize = 1.
 *              n_group > 1: E / n_group consecutive experts form a group, scored by
 *              the sum of its two best s + bias; only the topk_group best groups
 *              compete (DeepSeek-V3's routing).  A NaN adds nothing to its group's score, so
 *              that of one number and NaN is the number; a group of NaN alone ranks last.
 *   Every w is then multiplied by scale.  A NaN logit (or NaN score) ranks below
 *   -inf and has w = 0, -inf has w = 0, +inf counts as the largest finite value; a
 *   row with no finite logit gets w = 0 throughout, and ids that are still distinct.
 * offsets [E+1], tiles [E+1], order [T*k], place [T*k] int32: the grouping of the
 * picked pairs, all four or none (NULL); workspace then holds moe_group_workspace bytes.
 * 1 <= k <= E <= 4096, n_group <= 32, topk_group * (E / n_group) >= k.
 */
moe_status moe_route(int32_t T, int32_t E, int32_t k, int32_t logits_dtype, const void* logits, int32_t scoring,
                     const float* bias, int32_t n_group, int32_t topk_group, int32_t renormalize, float scale,
                     int32_t* topk_ids, float* topk_w, int32_t* offsets, int32_t* tiles, int32_t* order,
                     int32_t* place, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * The grouping alone, for ids from elsewhere.  An id outside [0, E) drops its pair:
 * place is -1, no row holds it, and the rows from offsets[E] on have order -1.
 */
moe_status moe_group_pairs(int32_t T, int32_t E, int32_t k, const int32_t* topk_ids, int32_t* offsets, int32_t* tiles,
                           int32_t* order, int32_t* place, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Matrix scales for NVFP4: g[i] = max |x_i| times the fp32 nearest to 1 / (6 * 448), of
 * each of G matrices of `count` elements (x in dtype MOE_BF16 or MOE_F32); 1 for a matrix
 * of zeros.  NaN or
 * infinity in a matrix gives that g.
 */
moe_status moe_fp4_scale(int32_t G, int64_t count, int32_t dtype, const void* x, float* g, void* stream);

/*
 * Quantise to 4 bits.  x in dtype MOE_BF16 or MOE_F32, K a multiple of 32.
 *   offsets NULL: x is a stack of G matrices [N, K]; row i of the output is row i of x.
 *   otherwise (G = 1): x [N / k, K], N = number of pairs; row t of x becomes the rows
 *   place[t, 0 .. k - 1] (none where -1), laid out by offsets / tiles [E + 1].
 * Per block, a = max |x|:
 *   NVFP4  block scale s = e4m3(a * r / g), r the fp32 nearest to 1 / 6, nearest even, at most
 *          448; code = e2m1(x / (s * g)).
 *   MXFP4  scale 2^X, X = floor(log2 a) - 2 within [-127, 127], 0 for a block of zeros;
 *          code = e2m1(x / 2^X).
 * Codes round to nearest, ties to even, and saturate at +-6 (infinities too).  A block
 * with a NaN gets the scale NaN.  Where s * g is 0 the codes are 0.  Every product and
 * division is a correctly rounded 32-bit one.  g: g_count = 1 or G fp32 scales, NULL = 1.
 */
moe_status moe_quantize_fp4(int32_t G, int32_t N, int32_t K, int32_t dtype, const void* x, int32_t wdtype,
                            const float* g, int32_t g_count, int32_t E, int32_t k, const int32_t* offsets,
                            const int32_t* tiles, const int32_t* place, uint8_t* codes, uint8_t* scales, void* stream);

/* The values e2m1(code) * (scale * g), in fp32, stored in dtype (MOE_BF16 or MOE_F32).
 * out [G, N, K], or [N, K] in expert order (offsets, tiles given; rows past offsets[E] are zero). */
moe_status moe_dequantize_fp4(int32_t G, int32_t N, int32_t K, int32_t wdtype, const uint8_t* codes,
                              const uint8_t* scales, const float* g, int32_t g_count, int32_t E,
                              const int32_t* offsets, const int32_t* tiles, int32_t dtype, void* out, void* stream);

/*
 * Products grouped by expert: out[i] = x_row(i) * w[e]^T for the rows i of each expert e.
 *   w [E, N, K] bf16; x [P, K] bf16 in expert order, or, with `order` and `place` given,
 *   [P / k, K] and grouped row i reads row order[i] / k.  K a multiple of 8.
 *   act 1: SwiGLU; w holds N/2 gate rows, then N/2 up rows (N a multiple of 32);
 *   out[i] = silu(gate) * up, N/2 columns.
 *   out [P, N or N/2] in out_dtype (MOE_BF16 or MOE_F32); rows from offsets[E] on are
 *   left as they are.
 *   Sums are fp32 in the tensor cores' accumulators, which truncate what is added to them.  A
 *   bf16 result is one such sum over K, rounded once (2e-6 off before that at K = 2000).  For an
 *   fp32 result the accumulators take K by 256 elements, and these sums are added up with
 *   rounding (2.5e-7 off, at K = 7168 too); its SwiGLU is within 11 half units of fp32.
 *   workspace: moe_grouped_matmul_workspace(P, E, K, order != NULL) bytes (0 or the rows
 *   gathered, for many rows per expert), 16-byte aligned.
 */
int64_t moe_grouped_matmul_workspace(int32_t P, int32_t E, int32_t K, int32_t gather);
moe_status moe_grouped_matmul(int32_t P, int32_t E, int32_t N, int32_t K, const void* x, int32_t x_rows, const int32_t* order,
                              const int32_t* place, int32_t k, const void* w, const int32_t* offsets, const int32_t* tiles, int32_t act,
                              int32_t out_dtype, void* out, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * The same with 4-bit rows and weights of one format (K a multiple of 32).  Products of
 * codes and block scales are summed in fp32, as above (an fp32 result: K by 1024 elements), then
 * multiplied by gx * gw[e] (gw_count = 1 or E; NULL = 1).  Their few bits leave such sums nearly
 * exact; where block scales differ widely (by e^2, K = 7168) they are 3e-6 off, for an fp32
 * result 5e-7.  out NULL: with act = 1 the result is quantised again as the 4-bit
 * rows out_codes / out_scales with matrix scale g_out (NULL = 1), and N/2 must be a multiple
 * of 32.  It is that of moe_quantize_fp4 on values with a bf16 result's sums and SwiGLU (silu
 * to |gate| + 10 units of 2^-23 of itself or 1e-18 of the gate), by products with reciprocals
 * good to three such units: a scale or code is another one where that carries a value over a
 * rounding edge.
 */
moe_status moe_grouped_matmul_fp4(int32_t P, int32_t E, int32_t N, int32_t K, int32_t wdtype, const uint8_t* x_codes,
                                  const uint8_t* x_scales, const float* gx, const uint8_t* w_codes,
                                  const uint8_t* w_scales, const float* gw, int32_t gw_count, const int32_t* offsets,
                                  const int32_t* tiles, int32_t act, int32_t out_dtype, void* out, uint8_t* out_codes,
                                  uint8_t* out_scales, const float* g_out, void* stream);

/*
 * out[t] = sum_j topk_w[t, j] * y[place[t, j]] in j order, fp32 sums, stored in
 * out_dtype.  y [P, N] in y_dtype; a pair with place -1 contributes nothing, and its
 * gate is not read into the sum.
 */
moe_status moe_combine(int32_t T, int32_t k, int32_t N, int32_t y_dtype, const void* y, const int32_t* place,
                       const float* topk_w, int32_t out_dtype, void* out, void* stream);

/* Synchronise `stream`; MOE_EDEVICE if a wait inside an operator kernel has run out on this
 * device since the last check (the flag is cleared). */
moe_status moe_operators_check(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPERATORS_H */
