/*
 * moe_mxfp4.h -- C ABI of the 4-bit experts of the GB300 (sm_103a) mixture-of-experts
 * library: the top-k router that makes the layer's routes, MXFP4 quantisation, the
 * grouped MXFP4 x MXFP4 product and the expert layer on MXFP4 weights.
 *
 * The conventions of moe_layer.h hold: device pointers owned by the caller and 16-byte
 * aligned (workspaces 256-byte aligned), nothing allocated, work enqueued on `stream`,
 * arguments checked on the host before anything is launched, its status codes, its
 * route tables, its treatment of expert ids outside [0, E) and its saturating binary16
 * outputs (a NaN stays a NaN).  Inference only: there is no backward pass.
 *
 * MXFP4 (OCP Microscaling Formats specification v1.0): elements are e2m1 (0, 0.5, 1, 1.5,
 * 2, 3, 4, 6 and their negatives; code bits: sign, two of exponent, one of mantissa), two
 * to a byte, the even element in the low nibble.  Every 32 consecutive elements of a row
 * share a scale byte b, an e8m0 number worth 2^(b - 127); b = 255 is NaN and makes the
 * 32 values NaN.  A block with largest magnitude a is quantised to
 *     b = max(floor(log2 a) - 2, -127) + 127   (0 for a = 0),
 *     element = x * 2^(127 - b) rounded to the nearest e2m1 value, ties to the even
 *     code, at most 6 in magnitude;
 * a block with an infinity or a NaN gets b = 255 and zero codes.
 */
#ifndef MOE_MXFP4_H
#define MOE_MXFP4_H

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of arrays that are not quantised. */
#define MOE_TYPE_F32 0
#define MOE_TYPE_F16 1
#define MOE_TYPE_BF16 2

/* ------------------------------------------------------------------------ */
/* Router                                                                    */
/* ------------------------------------------------------------------------ */

#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1

/*
 * The routes of M tokens from their gate logits.  Per token, with l_e its logits:
 *   p_e = exp(l_e - max l) / sum over e' of exp(l_e' - max l)    MOE_SCORE_SOFTMAX
 *   p_e = 1 / (1 + exp(-l_e))                                    MOE_SCORE_SIGMOID
 * The topK experts with the largest keys are chosen, in descending order of the key,
 * the lower expert first among equal ones.  The key is l_e (which orders as p_e does,
 * without its rounding), or p_e + bias[e] where a bias is given (a correction that
 * moves the choice, for balance, and not the weights).  The weights are
 *   probs[t][j] = scale * p_j, or with `renormalise` scale * p_j / (sum over the chosen).
 * A logit of -infinity or NaN masks its expert: it is never chosen and adds nothing to
 * a sum.  +infinity counts as the largest finite value.  Where fewer than topK experts
 * are left, the remaining slots get expert -1 (which the layer drops) and weight 0, and
 * weights whose sum is 0 are 0.
 *   logits [M][E] of `type` (MOE_TYPE_*), row t at element t * stride (stride >= E)
 *   bias   NULL or [E] fp32 (finite)
 *   expert_idx [M][topK], probs [M][topK]: what the layer takes
 * 1 <= topK <= E <= 1023, M >= 1, M * topK < 2^24.  All arithmetic is fp32.
 */
int32_t moe_route_topk(int32_t M, int32_t E, int32_t topK, const void* logits, int32_t type, int64_t stride,
                       const float* bias, int32_t score, int32_t renormalise, float scale, int32_t* expert_idx,
                       float* probs, void* stream);

/* ------------------------------------------------------------------------ */
/* Quantisation                                                              */
/* ------------------------------------------------------------------------ */

/*
 * Rows in MXFP4, the form the products take activations in:
 *   codes  [rows][D / 2] bytes
 *   scales [ceil(D / 128)][pitch] 32-bit words, pitch = rows rounded up to a multiple of 4:
 *          word [q][r] holds the scale bytes of elements 128 q .. 128 q + 127 of row r,
 *          the first 32 in its lowest byte (bytes past D, and words past the last row,
 *          are not read as scales of anything; quantisation writes 0 into the former).
 * D is a multiple of 32, 32 <= D <= 16384; 1 <= rows < 2^24.
 * moe_mxfp4_scale_words gives the words of `scales` (0 for other sizes).
 */
size_t moe_mxfp4_scale_words(int64_t rows, int32_t D);

/*
 * Quantises the M rows of x [M][D] (`type`, row t at element t * stride, stride >= D).
 *   row_map NULL: row t becomes row t (copies must be 1 and rows M).
 *   row_map [M][copies]: row t becomes every row row_map[t * copies + j] in [0, rows);
 *     other entries are skipped.  With the expanded_row_idx of moe_route_sort and
 *     copies = topK this is the dispatch to expert-major rows.  Rows that no entry
 *     names are not written.
 *   codes, scales: MXFP4 rows as above (`rows` of them).
 */
int32_t moe_mxfp4_quant(int32_t M, int32_t D, const void* x, int32_t type, int64_t stride, const int32_t* row_map,
                        int32_t copies, int32_t rows, uint8_t* codes, uint32_t* scales, void* stream);

/* The values MXFP4 rows stand for: out [rows][D] of `type`, rounded to nearest even and,
 * in binary16, saturated at +-65504. */
int32_t moe_mxfp4_dequant(int32_t rows, int32_t D, const uint8_t* codes, const uint32_t* scales, void* out,
                          int32_t type, void* stream);

/*
 * Weights in MXFP4.  W[E][N][D] (N output channels, a multiple of 128) is held as blocks
 * of 128 channels x 256 reduction steps, 17408 bytes each, that the products move with
 * one contiguous copy: block (e, nb, kb) is number (e * (N / 128) + nb) * KB + kb, KB =
 * ceil(D / 256).  In it
 *   - bytes 0 .. 16383: the codes; of channel r's 128 bytes of the step, the 16 bytes c
 *     (one scaled block of 32) are at r * 128 + (c ^ (r % 8)) * 16;
 *   - bytes 16384 + 512 q + 4 r + i (q < 2, i < 4): the scale byte of channel r's block
 *     c = 4 q + i.
 * Codes and scales past D are 0.  Channel r of block nb is channel nb * 128 + r of W, or
 * with gate_up (a GMM1 weight, whose first N / 2 channels are the gate and the others
 * the up projection) channel
 *     ((r / 32) % 2) * (N / 2) + nb * 64 + (r / 64) * 32 + r % 32:
 * 32 gate channels, the 32 up channels that multiply them, 32 gate, 32 up.
 * moe_mxfp4_weights_bytes gives the size (0 for sizes that are not supported).
 */
size_t moe_mxfp4_weights_bytes(int32_t E, int32_t N, int32_t D);

/* Quantises w [E][N][D] of `type` into blocks. */
int32_t moe_mxfp4_quant_weights(int32_t E, int32_t N, int32_t D, int32_t gate_up, const void* w, int32_t type,
                                uint8_t* blocks, void* stream);

/* Lays out weights that are MXFP4 already: codes [E][N][D / 2] and scale bytes
 * [E][N][D / 32], both 16-byte aligned, into blocks. */
int32_t moe_mxfp4_pack_weights(int32_t E, int32_t N, int32_t D, int32_t gate_up, const uint8_t* codes,
                               const uint8_t* scales, uint8_t* blocks, void* stream);

/* ------------------------------------------------------------------------ */
/* Grouped products                                                          */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace of the two products (0 for sizes that are not supported).  Its first
 * word is the status word that moe_workspace_status reads; each call clears it. */
size_t moe_mxfp4_gmm_workspace_size(int32_t R, int32_t E, int32_t N, int32_t D);

/*
 * c[d][n] = sum over k of a[d][k] * W[e][n][k] for every row d of expert e, rows
 * cumsum[e - 1] .. cumsum[e] - 1 (0 for e = 0) of the R expert-major rows; the sum in fp32,
 * rounded once to binary16.
 *   codes, scales  a in MXFP4 (R rows, depth D; moe_mxfp4_quant)
 *   cumsum [E]     inclusive prefix of the rows per expert, as moe_route_sort writes it
 *                  (entries are held to 0 .. R; rows >= cumsum[E-1] are not written)
 *   w              blocks of W[E][N][D], plain order
 *   c [R][N]       binary16
 * E <= 1023, N a multiple of 128 up to 65536, D as for rows.
 */
int32_t moe_mxfp4_gmm(int32_t R, int32_t E, int32_t N, int32_t D, const uint8_t* codes, const uint32_t* scales,
                      const int32_t* cumsum, const uint8_t* w, uint16_t* c, void* workspace, size_t workspace_bytes,
                      void* stream);

/*
 * The same product with N = 2 I channels in gate_up order, followed by SwiGLU and MXFP4
 * quantisation in the same kernel: with g and u the row's gate and up sums (fp32, not
 * rounded in between), h_i = g_i / (1 + exp(-g_i)) * u_i, written as MXFP4 rows
 *   h_codes [R][I / 2], h_scales (R rows, depth I).
 * I a multiple of 64 up to 8192.
 */
int32_t moe_mxfp4_gmm_swiglu(int32_t R, int32_t E, int32_t I, int32_t D, const uint8_t* codes, const uint32_t* scales,
                             const int32_t* cumsum, const uint8_t* w, uint8_t* h_codes, uint32_t* h_scales,
                             void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Whole layer                                                               */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace of moe_mxfp4_layer_fwd with up to d->M tokens, the other dimensions as they
 * are (0 if the dimensions are invalid). */
size_t moe_mxfp4_layer_workspace_size(const moe_dims_t* d);

/*
 * out[t, :] = sum over the token's valid routes of probs[t, j] * FFN_e(x[t, :]): the
 * expert layer of moe_layer_fwd on MXFP4 weights and activations.  x is quantised to
 * MXFP4, h = SwiGLU(GMM1) again, both products accumulate in fp32; the routes' rows are
 * weighted and added in fp32 too, and out is rounded to binary16 once.
 *   x, expert_idx, probs, out: as moe_layer_fwd (d->weight_layout is not read)
 *   w1  blocks of [E][2I][K] in gate_up order;  w2  blocks of [E][K][I], plain order
 *   workspace >= moe_mxfp4_layer_workspace_size of these dimensions, or of a larger M; its
 *              first word is the status word that moe_workspace_status reads.  Its contents on
 *              entry do not matter.
 * Up to 32 tokens and 256 routes (at sizes that fit the device) one kernel does most of
 * it, whose blocks wait for one another.  It is launched cooperatively, so it starts when
 * all of its blocks, one on every SM, can run beside what else is on the device.  On a stream
 * that may use fewer SMs than the device has, these calls take the path of the larger ones.
 */
int32_t moe_mxfp4_layer_fwd(const moe_dims_t* d, const uint16_t* x, const int32_t* expert_idx, const float* probs,
                            const uint8_t* w1, const uint8_t* w2, uint16_t* out, void* workspace,
                            size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Diagnostics                                                               */
/* ------------------------------------------------------------------------ */

/*
 * Exercises the wait of the few-token kernel's epilogue warps for their next unit of work, in a
 * block that has given up: one warp looks before the unit is there, three after.  They have to
 * answer alike, since they wait for one another afterwards: *answers (device int32 [4]) gets four
 * times 0 (given up).  Asynchronous on `stream`.
 */
int32_t moe_selftest_mxfp4_tickets(int32_t* answers, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MXFP4_H */
