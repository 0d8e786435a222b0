/*
 * fwt_experts.h - 8-bit integer products and products grouped by expert,
 * around the Walsh-Hadamard rotation, on MI355X (gfx950).
 *
 * Products of fwt_ffn.h's feed-forward block for models with experts, and for 8-bit
 * integers with one scale for a whole row (a token of activations, a channel
 * of weights), which leaves the sums of a product exact.  Four operators:
 *
 *   fwt_rotate_quantize_int8      x (I (x) H_b) as 8-bit integers and scales
 *   fwt_int8_matmul               the product of two such operands
 *   fwt_grouped_matmul            rows sorted by expert, each times its
 *                                 expert's weights, in 16 or 8 bits
 *   fwt_grouped_matmul_backward   its gradients, in 16 bits
 *
 * Groups.  `ends` is a device array of int32, one for each expert: expert e
 * has the rows from ends[e - 1] (from 0 for the first) up to ends[e], so equal
 * numbers are an expert without rows.  The device reads them when the call
 * runs; the host does not wait for them.  They are 0 .. m and do not fall;
 * numbers outside 0 .. m are cut to it.  Rows from ends[experts - 1] on belong to
 * no expert: they are not read.  Where ends fall, the results of rows that two
 * experts claim, or an expert and the rows of none, are unspecified, and dw of those
 * experts (nothing outside the arrays is read or written); all others hold.
 *
 * Conventions are fwt_ffn.h's: status codes, device buffers that the caller
 * owns, all arguments checked on the host before anything is enqueued, nothing
 * allocated, nothing synchronises, every call may be captured into a HIP
 * graph, sums have a fixed order, strides are in elements, last dimensions
 * are contiguous.  Sizes of 0 rows are no work and FWT_OK; k is at least 1.
 */
#ifndef QSE_FWT_EXPERTS_H
#define QSE_FWT_EXPERTS_H

#include "fwt_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The element type of 8-bit integers where an entry point below takes a type
 * (fwt_ffn_dtype for the others). */
#define FWT_INT8 5

/* codes, s = quantised y, y = x (I (x) H_bits) 2^(-bits/2).
 *  x           m x k (row stride ldx); bf16, f16 or fp32, at any alignment
 *              of its elements.
 *  bits        0 (no rotation) .. FWT_ROTATE_MAX_BITS; k is a multiple of
 *              2^bits.
 *  codes       m x k 8-bit integers -127 .. 127, row stride ldcodes >= k, a
 *              multiple of 16; 16-byte aligned.  Up to the next multiple of 16
 *              a row is padded with zeros.
 *  s           m floats, s = max(max |y| / 127, 2^-126) over the row; codes are
 *              y / s rounded to the nearest integer, of two the even one.  A
 *              row that holds a value that is not finite gets a NaN scale and
 *              zero codes; the others keep theirs.
 * Sums are in fp32, in an order that dtype, bits and k fix, the factor comes
 * after them: a sum past the fp32 range counts as not finite.  Rows of more
 * than 32768 elements are read twice.
 * FWT_EALIGN: codes or ldcodes misaligned; FWT_EINVAL: bits out of range or k
 * not a multiple of 2^bits; FWT_EUNSUPPORTED: 2^22 workgroups or more (one for
 * each row of more than 2048 elements, for four or more rows otherwise). */
int fwt_rotate_quantize_int8(const void* x, fwt_ffn_dtype dtype, int64_t m, int64_t k,
                             int64_t ldx, int bits, void* codes, int64_t ldcodes, float* s,
                             hipStream_t stream);

/* c[i][j] = a_scales[i] b_scales[j] sum_k a[i][k] b[j][k]: a is m x k and b
 * n x k 8-bit integers (-128 is one of them), c bf16, f16 or fp32.  The sum is
 * exact in 32-bit integers: k is below 2^17 (FWT_EUNSUPPORTED).  It is rounded
 * to fp32, times a_scales[i], times b_scales[j], and then to c's type; so where
 * a scale is NaN the results are, and no other.  A row of a or b is read up to k
 * only, whatever its padding holds.  The strides lda and ldb are multiples of
 * 16 below 2^23, a and b 16-byte aligned (FWT_EALIGN; a longer stride, or more
 * than 2^22 tiles of 128 x 64 results, FWT_EUNSUPPORTED).
 *  ws          scratch of fwt_int8_matmul_workspace bytes (0 for most sizes),
 *              16-byte aligned, one for each call that may run at the same
 *              time: a long contraction with few results is then shared by
 *              several workgroups.  NULL: it is not shared, which takes
 *              longer.  The results are the same, bit for bit. */
int fwt_int8_matmul_workspace(int64_t m, int64_t n, int64_t k, fwt_ffn_dtype ctype,
                              size_t* bytes);
int fwt_int8_matmul(const void* a, int64_t lda, const float* a_scales, const void* b,
                    int64_t ldb, const float* b_scales, int64_t m, int64_t n, int64_t k, void* c,
                    fwt_ffn_dtype ctype, int64_t ldc, void* ws, size_t ws_bytes,
                    hipStream_t stream);

/* y[i][j] = sum_k x[i][k] w[e][j][k] for the rows i of expert e: x is m x k,
 * w experts x n x k (ldw between rows, stride_w between experts), y m x n.
 *  dtype       FWT_BF16 or FWT_F16: y has the same type, the scales are NULL;
 *              sums are in fp32 and only y is rounded; any alignment (operands
 *              whose addresses and strides are multiples of 16 bytes are read
 *              faster) and row strides below 2^22.  FWT_INT8: y bf16, f16 or
 *              fp32 with x_scales (m) and w_scales (experts x n, contiguous),
 *              as fwt_int8_matmul computes it; k below 2^17, x, w and their
 *              strides 16-byte aligned, row strides below 2^23.
 *  zero_rest   the rows of y that belong to no expert: 0 leaves them as they
 *              were, otherwise they become 0.
 *  ws          scratch of fwt_grouped_matmul_workspace_for bytes (0 for most
 *              sizes), as for fwt_int8_matmul, and for copies of 16-bit operands
 *              that are misaligned (up to 1 GiB) where k is no multiple of 8 and a
 *              large call on aligned rows takes less time with the copying.  NULL:
 *              nothing is shared or copied, which takes longer and may add fp32 sums
 *              in another order.
 *              fwt_grouped_matmul_workspace: enough for any operands of the sizes;
 *              .._for: of x and w, of which the addresses and strides count and
 *              nothing is read.
 * Which kernel runs, and so the order of fp32 sums, goes by the sizes, the
 * addresses' alignment and ws, not by where the groups end.
 * More than 2^22 tiles of 128 x 64 results (every expert may have one row of
 * tiles that is not whole), or more than 2^16 experts, are FWT_EUNSUPPORTED. */
int fwt_grouped_matmul_workspace(int dtype, int64_t experts, int64_t m, int64_t n, int64_t k,
                                 size_t* bytes);
int fwt_grouped_matmul_workspace_for(const void* x, int64_t ldx, const void* w, int64_t ldw,
                                     int64_t stride_w, int64_t experts, int dtype, int64_t m,
                                     int64_t n, int64_t k, size_t* bytes);
int fwt_grouped_matmul(const void* x, int64_t ldx, const float* x_scales, const void* w,
                       int64_t ldw, int64_t stride_w, const float* w_scales,
                       const int32_t* ends, int64_t experts, int dtype, int64_t m, int64_t n,
                       int64_t k, void* y, fwt_ffn_dtype ytype, int64_t ldy, int zero_rest,
                       void* ws, size_t ws_bytes, hipStream_t stream);

/* Gradients of fwt_grouped_matmul on bf16 or f16 for dy (m x n):
 *   dx[i] = dy[i] w[e]  for the rows i of expert e (0 for rows of no expert),
 *   dw[e] = sum over e's rows i of dy[i]^T x[i]  (0 for an expert without rows),
 * dx m x k, dw experts x n x k (lddw between rows, stride_dw between experts).
 * Sums are in fp32 and only the results are rounded.  All arrays have the dtype,
 * any alignment, row strides below 2^22.  dx or dw may be NULL: that gradient is
 * not computed.  ws: scratch of fwt_grouped_matmul_backward_workspace_for bytes
 * (dx, dw: not 0 for a gradient that is wanted), or of .._workspace, as above. */
int fwt_grouped_matmul_backward_workspace(int64_t experts, int64_t m, int64_t n, int64_t k,
                                          size_t* bytes);
int fwt_grouped_matmul_backward_workspace_for(const void* x, int64_t ldx, const void* w,
                                              int64_t ldw, int64_t stride_w, int64_t experts,
                                              const void* dy, int64_t lddy, int64_t m, int64_t n,
                                              int64_t k, int dx, int dw, size_t* bytes);
int fwt_grouped_matmul_backward(const void* x, int64_t ldx, const void* w, int64_t ldw,
                                int64_t stride_w, const int32_t* ends, int64_t experts,
                                const void* dy, int64_t lddy, fwt_ffn_dtype dtype, int64_t m,
                                int64_t n, int64_t k, void* dx, int64_t lddx, void* dw,
                                int64_t lddw, int64_t stride_dw, void* ws, size_t ws_bytes,
                                hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QSE_FWT_EXPERTS_H */
