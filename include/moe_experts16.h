/*
 * moe_experts16.h -- C ABI of the 16-bit experts of the GB300 (sm_103a) mixture-of-experts
 * library: products grouped by expert on binary16 or bfloat16 weights, SwiGLU, the dispatch
 * and combine of rows, each with its gradient, and the low-rank adapters of many requests.
 *
 * The conventions of moe_layer.h hold: device pointers owned by the caller and 16-byte
 * aligned (workspaces 256-byte aligned), dense row-major arrays, nothing allocated, work
 * enqueued on `stream`, arguments checked on the host before anything is launched, its
 * status codes and its route tables.  Calls that may overlap on the device (on streams of
 * their own, or as graphs replayed at once) need workspaces of their own.  `type` is MOE_TYPE_F16 or MOE_TYPE_BF16 and is the
 * type of every array whose type is not named.  Sums are held in fp32 and rounded to
 * nearest even where they are stored, once; binary16 saturates at +-65504 (a NaN stays a
 * NaN), bfloat16 overflows to infinity.  The tensor cores' fp32 sums drop bits towards
 * zero: of n products 2^-27 n of their magnitudes at most.  n is the depth of a product
 * or of a gradient for the rows (that is half a step of binary16 at the deepest, 65536, a
 * sixteenth of it at 4096; bfloat16 an eighth of those), and for a weight gradient of any
 * number of rows at most 4096 (binary16) or 32768 (bfloat16), in fp32 512 or 768: longer
 * sums are made of such parts, added in fp32.
 *
 * In binary16 an infinity that comes in is stored as +-65504 too, by the gradients as well: a
 * loss scaler that looks for infinities finds none in da, dgu, dy or a 16-bit dw, and an fp32 dw
 * made of those is finite.  It has to look at what it passes in, at dprobs and fp32 sums of
 * its own, or take +-65504 for an overflow.  (bfloat16 keeps infinities.)
 *
 * A batch without rows (R, M or rows 0) is refused: MOE_ERR_SHAPE, nothing written.  The caller
 * leaves the call out, and clears a dw that it does not accumulate into.
 *
 * Expert-major rows: those of expert e are cumsum[e - 1] .. cumsum[e] - 1 (from 0 for
 * e = 0) of R rows; cumsum [E] is the inclusive prefix that moe_route_sort writes (entries
 * are held to 0 .. R).  Rows from cumsum[E - 1] on belong to no expert: outputs there are
 * left as they were, and what inputs hold there (NaN too) reaches nothing.
 *
 * A training step through the layer, with x [M][K], routes from moe_route_sort:
 *   a = dispatch16(x);  gu = gmm16(a, w1);  h = swiglu16(gu);  y = gmm16(h, w2);
 *   out = combine16(y, probs)
 * and back, from dout:
 *   dy, dprobs = combine16_grad(dout, y, probs);
 *   dh = gmm16_input_grad(dy, w2);  dw2 = gmm16_weight_grad(dy, h);
 *   dgu = swiglu16_grad(dh, gu);
 *   da = gmm16_input_grad(dgu, w1);  dw1 = gmm16_weight_grad(dgu, a);
 *   dx = combine16(da, probs NULL)
 */
#ifndef MOE_EXPERTS16_H
#define MOE_EXPERTS16_H

#include "moe_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------ */
/* Products grouped by expert                                                */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace of the three products (0 for sizes that are not supported).  Its first
 * word is the status word that moe_workspace_status reads; each call clears it.
 * 1 <= R < 2^24, 1 <= E <= 1023; N and D are multiples of 8, from 8 to 65536. */
size_t moe_gmm16_workspace_size(int32_t R, int32_t E, int32_t N, int32_t D);

/*
 * c[d][n] = sum over k of a[d][k] * w[e][n][k] for every row d of expert e.
 *   a [R][D], w [E][N][D], c [R][N].  With E = 1 and cumsum[0] = R a plain projection.
 */
int32_t moe_gmm16(int32_t R, int32_t E, int32_t N, int32_t D, int32_t type, const void* a, const int32_t* cumsum,
                  const void* w, void* c, void* workspace, size_t workspace_bytes, void* stream);

/* Its gradient for the rows: da[d][k] = sum over n of dc[d][n] * w[e][n][k].
 *   dc [R][N], w [E][N][D], da [R][D]. */
int32_t moe_gmm16_input_grad(int32_t R, int32_t E, int32_t N, int32_t D, int32_t type, const void* dc,
                             const int32_t* cumsum, const void* w, void* da, void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * Its gradient for the weights: dw[e][n][k] = sum over the rows d of expert e of
 * dc[d][n] * a[d][k]; 0 for an expert without rows.
 *   dc [R][N], a [R][D], dw [E][N][D] of dw_type: `type` or MOE_TYPE_F32.
 *   accumulate: the sum is added to what dw holds (MOE_TYPE_F32 only: a running sum is not
 *   kept in 16 bits).
 */
int32_t moe_gmm16_weight_grad(int32_t R, int32_t E, int32_t N, int32_t D, int32_t type, const void* dc, const void* a,
                              const int32_t* cumsum, void* dw, int32_t dw_type, int32_t accumulate, void* workspace,
                              size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* SwiGLU                                                                    */
/* ------------------------------------------------------------------------ */

/*
 * h[d][i] = g s(g) u with g = gu[d][i], u = gu[d][I + i], s(g) = 1 / (1 + exp(-g)), for the
 * rows d below cumsum[E - 1].
 *   gu [R][2I], h [R][I]; I a multiple of 8 from 8 to 32768.
 */
int32_t moe_swiglu16(int32_t R, int32_t E, int32_t I, int32_t type, const void* gu, const int32_t* cumsum, void* h,
                     void* stream);

/*
 * Its gradient: with dh [R][I],
 *   dgu[d][i] = dh u s(g) (1 + g (1 - s(g))),   dgu[d][I + i] = dh g s(g).
 *   dgu [R][2I], which may be gu itself.
 *   h   NULL, or [R][I]: gets what moe_swiglu16 gives, so that it need not be kept for the
 *       weight gradient of the product behind it.  It may be dh itself.
 */
int32_t moe_swiglu16_grad(int32_t R, int32_t E, int32_t I, int32_t type, const void* dh, const void* gu,
                          const int32_t* cumsum, void* dgu, void* h, void* stream);

/* ------------------------------------------------------------------------ */
/* Dispatch and combine                                                      */
/* ------------------------------------------------------------------------ */

/* row_map [M][copies] names rows in [0, rows): expanded_row_idx of moe_route_sort with
 * copies = topK.  Other entries (-1: a dropped route) are skipped.
 * 1 <= M, rows < 2^24; M * copies < 2^24; D a multiple of 8 from 8 to 65536. */

/* out[row_map[t][j]] = x[t].  x [M][D], out [rows][D]; rows that no entry names are left as
 * they were.  Entries of one row twice have to be of the same token. */
int32_t moe_dispatch16(int32_t M, int32_t D, int32_t copies, int32_t rows, int32_t type, const void* x,
                       const int32_t* row_map, void* out, void* stream);

/* out[t] = sum over j of probs[t][j] * y[row_map[t][j]], added in the order of j; without
 * routes 0.  y [rows][D], probs [M][copies] fp32 or NULL (all 1: the gradient of
 * moe_dispatch16), out [M][D]. */
int32_t moe_combine16(int32_t M, int32_t D, int32_t copies, int32_t rows, int32_t type, const void* y,
                      const int32_t* row_map, const float* probs, void* out, void* stream);

/*
 * The gradient of moe_combine16 for y and probs:
 *   dy[row_map[t][j]] = probs[t][j] * dout[t],   dprobs[t][j] = <dout[t], y[row_map[t][j]]>.
 *   dout [M][D], y [rows][D], dy [rows][D] (rows that no entry names are left as they were;
 *   it may be y itself), dprobs [M][copies] fp32, 0 for entries that are skipped.
 * No row may be named twice.
 */
int32_t moe_combine16_grad(int32_t M, int32_t D, int32_t copies, int32_t rows, int32_t type, const void* dout,
                           const void* y, const int32_t* row_map, const float* probs, void* dy, float* dprobs,
                           void* stream);

/* ------------------------------------------------------------------------ */
/* Low-rank adapters                                                         */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace of moe_lora16 (0 for sizes that are not supported).
 * 1 <= M < 2^24; N and D multiples of 8 from 8 to 65536; rank a multiple of 8 from 8 to 128
 * (adapters of a lower rank are padded with zeros). */
size_t moe_lora16_workspace_size(int32_t M, int32_t N, int32_t D, int32_t rank);

/*
 * Adapters of many requests beside a projection that they share:
 *   out[t] = base[t] + scales[l] * b[l] (a[l] x[t])
 * with l the adapter of token t; out[t] = base[t] for a token without one.
 *   x [M][D]; base [M][N], what the projection gave; out [M][N], which may be base itself
 *   route [M], cumsum [L]: the tokens sorted by adapter, sorted_src_route and cumsum of
 *       moe_route_sort on the tokens' adapters (topK = 1, E = L; an id outside [0, L) is no
 *       adapter).  Made once, they serve every projection of a batch.  Entries of route
 *       outside [0, M) are skipped; no token may be there twice.
 *   a [L][rank][D], b [L][N][rank]; scales [L] fp32 or NULL (all 1)
 * The rank values of a token between the two products keep 16 significant bits.
 */
int32_t moe_lora16(int32_t M, int32_t N, int32_t D, int32_t rank, int32_t L, int32_t type, const void* x,
                   const int32_t* route, const int32_t* cumsum, const void* a, const void* b, const float* scales,
                   const void* base, void* out, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS16_H */
