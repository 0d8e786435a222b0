/*
 * fwt_ffn.h - the feed-forward block around the Walsh-Hadamard rotation, in
 * 8 and 16 bits, on MI355X (gfx950).
 *
 * A rotation by H_b spreads a few large channels of an activation over all
 * of them before its values are rounded to 8 bits; rotated weights undo it:
 * (x H)(W H)^T = x W^T.  Four operators, used one after another:
 *
 *   fwt_rotate_quantize   x (I (x) H_b) as e4m3 codes and scales
 *   fwt_scaled_matmul     the product of two operands of codes and scales
 *   fwt_gated_ffn         act(x Wg^T) * (x Wu^T)
 *   fwt_gated_ffn_backward   its gradients
 *
 * Scales.  Along the contraction axis k every 128 elements share one: of one
 * row (FWT_SCALES_ROW: a float array [ceil(k/128)][rows]) or of a tile of
 * 128 rows (FWT_SCALES_TILE: [ceil(k/128)][ceil(rows/128)]), contiguous.
 * The value of a code is code * scale.
 *
 * Conventions are fwt.h's: its status codes, device buffers that the caller
 * owns, on the calling thread's current device; the stream is one of that
 * device; all arguments are checked on the host before anything is enqueued
 * (FWT_EINVAL for a null pointer, a size or stride out of range, buffers
 * that are not device memory of the needed size, and one that is written
 * and lies, from its first element to its last, across another's; inputs
 * may be the same); nothing is
 * allocated and nothing synchronises, so every call may be captured into a
 * HIP graph.  Results do not depend on what else runs: sums have a fixed
 * order.  Strides are in elements, last dimensions are contiguous.  Sizes of
 * 0 rows (m or n) are no work and FWT_OK; k must be at least 1.
 */
#ifndef QSE_FWT_FFN_H
#define QSE_FWT_FFN_H

#include "fwt.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FWT_BF16 = 0, FWT_F16 = 1, FWT_FP32 = 2, FWT_E4M3 = 3 } fwt_ffn_dtype;
typedef enum { FWT_SCALES_ROW = 0, FWT_SCALES_TILE = 1 } fwt_scales;
/* silu: g / (1 + e^-g); gelu: g times the normal distribution function. */
typedef enum { FWT_SILU = 0, FWT_GELU = 1 } fwt_activation;

/* Largest rotation: 2^FWT_ROTATE_MAX_BITS elements, of a transposed input
 * 2^FWT_ROTATE_MAX_BITS_T. */
#define FWT_ROTATE_MAX_BITS 14
#define FWT_ROTATE_MAX_BITS_T 7

/* codes, scales = quantised y, y = x (I (x) H_bits) 2^(-bits/2).
 *  x           m x k (row stride ldx), or with `transposed` k x m; bf16,
 *              f16 or fp32, at any alignment of its elements.
 *  bits        0 (no rotation) .. 14, or .. 7 with `transposed`; k is a
 *              multiple of 2^bits.
 *  codes       m x k e4m3 (the OCP format without infinities), row stride
 *              ldcodes >= k, a multiple of 16; 16-byte aligned.  Up to the
 *              next multiple of 16 a row is padded with zeros.
 *  scales      as fwt_scales says, s = max(max |y| / 448, 2^-126) over the
 *              block; codes are y / s rounded to nearest even.  A block that
 *              holds a value that is not finite gets a NaN scale and NaN
 *              codes; the others keep theirs.
 *  ws          scratch of fwt_rotate_quantize_workspace bytes (0 except for
 *              tile scales with bits > 7), 16-byte aligned; two calls that
 *              may run at the same time need one each.
 * Sums are in fp32, in an order that dtype and bits fix, the factor comes
 * after them: a sum past the fp32 range counts as not finite.
 * FWT_EALIGN: codes, ldcodes or ws misaligned; FWT_EINVAL: bits out of
 * range or k not a multiple of 2^bits; FWT_EUNSUPPORTED: 2^29 blocks of 128
 * or more, or of a transposed input or with tile scales more than 65535 * 128
 * rows or 2^22 blocks in one. */
int fwt_rotate_quantize_workspace(int64_t m, int64_t k, int bits, fwt_scales scales,
                                  int transposed, size_t* bytes);
int fwt_rotate_quantize(const void* x, fwt_ffn_dtype dtype, int64_t m, int64_t k, int64_t ldx,
                        int transposed, int bits, fwt_scales scales, void* codes,
                        int64_t ldcodes, float* s, void* ws, size_t ws_bytes,
                        hipStream_t stream);

/* c[i][j] = sum_k a[i][k] b[j][k]: a is m x k codes with row scales, b is
 * n x k codes with scales of either kind, c bf16, f16 or fp32.  Sums are in
 * 32 bits; the product of two scales, rounded to fp32, multiplies their block's
 * 128-element sum (so it has to be a normal fp32 number).  For f16 and
 * fp32 the products go through the 16-bit matrix instruction, which keeps all
 * of them.  For bf16 they go through the 8-bit one at twice the rate, which
 * cuts each towards zero to a step of 2^-13 of the largest of 8 neighbours
 * along k: together at most 7 * 2^-13 of that largest one, a fifth of bf16's
 * rounding where all products have one sign.  A row of a
 * or b is read up to k only, whatever its padding holds.  The strides lda
 * and ldb are multiples of 16 below 2^23, a and b 16-byte aligned
 * (FWT_EALIGN; a longer stride, or more than 2^22 tiles of 128 x 64 results,
 * FWT_EUNSUPPORTED).
 *  ws          scratch of fwt_scaled_matmul_workspace bytes (0 for most
 *              sizes), 16-byte aligned, one for each call that may run at the
 *              same time: a long contraction with few results is then shared
 *              by several workgroups, whose sums a second kernel adds in a
 *              fixed order.  NULL: it is not shared, which takes longer and
 *              adds in another order. */
int fwt_scaled_matmul_workspace(int64_t m, int64_t n, int64_t k, fwt_scales b_kind,
                                fwt_ffn_dtype ctype, size_t* bytes);
int fwt_scaled_matmul(const void* a, int64_t lda, const float* a_scales, const void* b,
                      int64_t ldb, const float* b_scales, fwt_scales b_kind, int64_t m,
                      int64_t n, int64_t k, void* c, fwt_ffn_dtype ctype, int64_t ldc,
                      void* ws, size_t ws_bytes, hipStream_t stream);

/* h = act(x gate^T) * (x up^T): x is m x k, gate and up n x k, of one
 * dtype.  bf16 and f16: h has the same dtype, the scales are NULL; any
 * alignment (operands whose addresses and strides are multiples of 16 bytes
 * are read faster) and strides below 2^22.  e4m3: x_scales row scales, gate_scales and up_scales
 * tile scales, alignment as for fwt_scaled_matmul, h bf16, f16 or fp32.
 * Both products are summed as fwt_scaled_matmul sums them, in 32 bits, and
 * only h is rounded.  ws: as there, of fwt_gated_ffn_workspace bytes. */
int fwt_gated_ffn_workspace(fwt_ffn_dtype dtype, int64_t m, int64_t n, int64_t k,
                            fwt_ffn_dtype htype, size_t* bytes);
int fwt_gated_ffn(const void* x, int64_t ldx, const float* x_scales, const void* gate,
                  int64_t ldgate, const float* gate_scales, const void* up, int64_t ldup,
                  const float* up_scales, fwt_ffn_dtype dtype, int64_t m, int64_t n, int64_t k,
                  fwt_activation act, void* h, fwt_ffn_dtype htype, int64_t ldh, void* ws,
                  size_t ws_bytes, hipStream_t stream);

/* Gradients of fwt_gated_ffn on bf16 or f16 for dh (m x n):
 *   dx = dg gate + du up,  dgate = dg^T x,  dup = du^T x,
 *   dg = dh * up' * act'(g),  du = dh * act(g),  g = x gate^T, up' = x up^T.
 * g and up' are computed again in 32 bits, not stored by the forward pass;
 * dg and du are rounded to the dtype once for the matrix products, as a
 * program that stores them would (bf16: the gradients' error in norm is about
 * sqrt(2) of their own rounding's).  f16: where the largest finite one is above
 * 65504 or below 2^-12 both are stored times a power of two that the products
 * take out again, so they lose bits only below 2^-29 of the largest (otherwise
 * below 2^-14) and the gradients overflow only where they are past the type's
 * range themselves.  All arrays have the dtype; ldx, ldgate and ldup are below 2^22, n below 2^21 and the
 * three products have fewer than 2^22 tiles (FWT_EUNSUPPORTED).  ws: scratch of fwt_gated_ffn_backward_workspace bytes,
 * 16-byte aligned, one for each call that may run at the same time. */
int fwt_gated_ffn_backward_workspace(int64_t m, int64_t n, int64_t k, size_t* bytes);
int fwt_gated_ffn_backward(const void* x, int64_t ldx, const void* gate, int64_t ldgate,
                           const void* up, int64_t ldup, const void* dh, int64_t lddh,
                           fwt_ffn_dtype dtype, int64_t m, int64_t n, int64_t k,
                           fwt_activation act, void* dx, int64_t lddx, void* dgate,
                           int64_t lddgate, void* dup, int64_t lddup, void* ws,
                           size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QSE_FWT_FFN_H */
