/*
 * nf4_int8.h -- C ABI of the products in 8-bit integers of libnf4.so: linear
 * layers whose weight is held as int8 with one scale for each output channel
 * and whose activations are quantised with one scale for each token, multiplied
 * on the integer matrix cores; plain, and for stacks of experts.  They stand beside
 * the blockwise 8-bit formats of nf4.h, which multiply in bf16.
 *
 * Conventions (memory, streams, errors, status codes) are those of nf4.h: all
 * pointers are device memory of the caller, work is enqueued asynchronously
 * on `stream`, nothing is allocated, freed or retained, an error enqueues
 * nothing.  Sums of products are exact (32-bit integers), so repeated calls on the
 * same inputs give bitwise identical outputs.  Every call can be captured into a
 * HIP graph.  Written tensors are contiguous and overlap nothing that the call
 * reads.
 *
 * Rows of integers.  A row of K values is kept in nf4_int8_row_bytes(K) bytes (K
 * rounded up to a multiple of 128), the bytes behind K zero, with one fp32 scale:
 *   top = max |x|;  scale = fp32(top / 127);  q = 127 x / top to the nearest
 *   integer, half-way to even (no rounding before that one)
 * so q lies in -127 .. 127 and stands for q * scale.  A row with top < 2^-119 is
 * kept as zeros (scale 0); one that holds a NaN or an infinity is kept as NaN
 * (scale NaN, q 0).  Weights are such rows too, one for each output channel.
 *
 * Limits (else NF4_ERR_UNSUPPORTED).  K is at most 130944, so that no sum of K
 * products of bytes passes 32 bits; M and total_M are at most 2^28, N at most
 * 2^28, E at most 1024, and a launch holds fewer than 2^32 threads.
 */
#ifndef NF4_INT8_H_
#define NF4_INT8_H_

#include "nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define NF4_DTYPE_I8 2  /* for x of the products: rows as nf4_int8_quantize leaves them */

/* Bytes of a row of K integers (negative for K < 0). */
int64_t nf4_int8_row_bytes(int64_t K);

/* nf4_int8_quantize -- x [M, K] (NF4_DTYPE_F32 or NF4_DTYPE_BF16, rows `stride`
 * elements apart) to q int8 [M, nf4_int8_row_bytes(K)] (16-byte aligned) and scale
 * f32 [M]. */
int nf4_int8_quantize(const void* x, int dtype, int64_t stride, int64_t M, int64_t K,
                      int8_t* q, float* scale, void* stream);

/*
 * nf4_int8_matmul -- y[m, n] = fp32(sum_k xq[m, k] q[n, k]) * scale[n] * x_scale[m] + bias[n],
 * in fp32, rounded once to y_dtype (F32 or BF16).
 *   x        [M, K] F32 or BF16, rows `stride` elements apart, quantised on the
 *            way; or NF4_DTYPE_I8 rows with x_scale (stride is then not read)
 *   q, scale weight [N, K] as nf4_int8_quantize leaves it
 *   bias     f32 [N] or NULL
 *   ws       nf4_int8_workspace(x_dtype, M, M, N, K, 0) bytes, 16-byte aligned
 */
int nf4_int8_matmul(const void* x, int x_dtype, int64_t stride, const float* x_scale,
                    int64_t M, const int8_t* q, const float* scale, int64_t N,
                    int64_t K, const float* bias, void* y, int y_dtype, void* ws,
                    size_t ws_bytes, void* stream);

/*
 * nf4_int8_grouped_matmul -- the same for a stack of experts over expert-sorted
 * rows: y [total_M, N], rows offsets[e] .. offsets[e+1]-1 through expert e.
 *   x        [x_rows, K] as above.  tokens int32 [total_M] names the row of x for
 *            each row of y (nothing is gathered in memory); NULL: row r reads row
 *            r, and x_rows is total_M
 *   offsets  int32 [E + 1], non-decreasing from 0 to at most total_M; entries
 *            are clamped, and so are tokens, so malformed arrays give wrong rows
 *            but no access out of range
 *   q, scale the stack [E, N, K] quantised as E*N rows
 * Rows behind offsets[E] are written as zeros where fill_outside is 1 and left as
 * they were where it is 0; their tokens are not read.  (Without tokens such rows of x are
 * quantised with the others; no result depends on them.)
 *   ws       nf4_int8_workspace(x_dtype, x_rows, total_M, N, K, E) bytes
 */
int nf4_int8_grouped_matmul(const void* x, int x_dtype, int64_t stride,
                            const float* x_scale, int64_t x_rows, const int32_t* tokens,
                            const int32_t* offsets, int32_t E, int64_t total_M,
                            const int8_t* q, const float* scale, int64_t N, int64_t K,
                            void* y, int y_dtype, int fill_outside, void* ws,
                            size_t ws_bytes, void* stream);

/* Workspace bytes of the products on the current device (E 0: the plain one);
 * SIZE_MAX for sizes they refuse.  A workspace belongs to one call at a time. */
size_t nf4_int8_workspace(int x_dtype, int64_t x_rows, int64_t M, int64_t N, int64_t K,
                          int32_t E);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* NF4_INT8_H_ */
