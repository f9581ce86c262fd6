/*
 * token_ops.h -- C ABI of libconv3d.so for what follows a convolutional patch
 * embedding: rows of tokens, normalised or activated and brought to 8 bits
 * with one scale per token, and the matrix product of such rows with 8-bit
 * weights that have one scale per output channel.
 *
 *   rms_norm_quant_fwd   h = x + residual;  v = h / sqrt(mean(h^2) + eps) * weight
 *   act_quant_fwd        v = act(x), or act(gate) * value for x = [gate | value]
 *     both:              scale = max|v| / qmax over the token's row,
 *                        q = the nearest code of v / scale (qmax: 127 int8, 448 e4m3)
 *   linear_w8a8_fwd      out[m,n] = act(scale_x[m] * scale_w[n] *
 *                                       sum_k x[m,k] w[n,k] + bias[n])
 *
 * Conventions (status codes, conv_last_error, streams and ownership are
 * those of conv3d.h):
 *   - A matrix is rows of contiguous elements; `*_stride` is the distance
 *     between rows in elements (at least the row's length).  Pointers need
 *     the alignment of their element type only.  Rows that are 16-byte
 *     aligned take the wider paths.
 *   - Everything between the inputs and the outputs is held in 32 bits: h is
 *     rounded only where residual_out stores it (v is computed from the
 *     unrounded h).
 *   - A row of zeros gets scale 1 and codes 0 (whatever eps is: the norm of
 *     zeros is zeros).  A row whose v holds a NaN or an infinity, or whose mean
 *     square is beyond fp32, gets scale NaN and codes 0, so that everything
 *     computed from it is NaN rather than a finite value that means nothing.
 *     SiLU and GELU of -inf are NaN (a product with 0), relu's is 0.
 *   - act_quant_fwd's SiLU and GELU hold their relative accuracy in the negative
 *     tail down to 2^-119; what is smaller may count as 0.
 *   - Zero tokens (and zero outputs of the product) are valid and launch
 *     nothing.  A width of zero is CONV_ERR_INVALID.
 */
#ifndef TOKEN_OPS_GB300_H
#define TOKEN_OPS_GB300_H

#include "conv3d.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types beside conv_dtype's CONV_DTYPE_BF16 and CONV_DTYPE_FP8_E4M3. */
enum { CONV_DTYPE_INT8 = 2, CONV_DTYPE_F16 = 3, CONV_DTYPE_F32 = 4 };

/* The root-mean-square norm of tokens x [tokens, width], with an optional
 * residual added first, quantised per token.
 *   x, x_dtype         BF16, F16 or F32
 *   residual           NULL, or rows of res_dtype: x's type or F32
 *   weight             [width], weight_dtype x's type or F32; NULL: ones
 *   q, q_dtype         codes, INT8 or FP8_E4M3; scale: fp32 [tokens]
 *   residual_out       NULL, or (only with a residual) rows of res_dtype that
 *                      receive h; may be `residual` itself, or x where it has
 *                      res_dtype: each element is read before it is written.
 *                      Any other overlap of inputs and outputs is undefined. */
int rms_norm_quant_fwd(const void* x, int x_dtype, int64_t x_stride, const void* residual,
                       int res_dtype, int64_t res_stride, const void* weight, int weight_dtype,
                       float eps, int64_t tokens, int64_t width, int q_dtype, void* q,
                       int64_t q_stride, float* scale, void* residual_out,
                       int64_t res_out_stride, cudaStream_t stream);

/* The activation of tokens, quantised per token.  `act` is one of conv3d.h's
 * CONV_ACT_*.  gated != 0: x has 2*width columns, v = act(first half) *
 * second half; otherwise v = act(x) (with CONV_ACT_NONE this quantises rows
 * as they are: activations, or weights per output channel). */
int act_quant_fwd(const void* x, int x_dtype, int64_t x_stride, int act, int gated,
                  int64_t tokens, int64_t width, int q_dtype, void* q, int64_t q_stride,
                  float* scale, cudaStream_t stream);

/* The product of tokens x [tokens, width] and weights w [outputs, width],
 * both of `dtype` (INT8 or FP8_E4M3), with fp32 scales [tokens] and
 * [outputs] (NULL: ones), an optional fp32 bias [outputs] and an activation.
 * out: BF16, F16 or F32, [tokens, outputs].  The activations keep their relative
 * accuracy in the negative tail in each of them; SiLU and GELU of -inf are NaN.
 * Sums are fp32: exact for int8 while every partial sum stays within 2^24
 * (any width up to 1024, and wider ones unless nearly all products are at
 * the type's limits with one sign), within a relative 2^-23 per 16 products
 * beyond.
 * workspace: linear_w8a8_workspace_size bytes, 16-byte aligned; NULL if that
 * is 0. */
int linear_w8a8_fwd(const void* x, int64_t x_stride, const void* w, int64_t w_stride, int dtype,
                    int64_t tokens, int64_t outputs, int64_t width, const float* scale_x,
                    const float* scale_w, const float* bias, int act, void* out, int out_dtype,
                    int64_t out_stride, void* workspace, size_t workspace_bytes,
                    cudaStream_t stream);

/* Up to this many tokens linear_w8a8_fwd needs no workspace. */
#define LINEAR_W8A8_NO_WORKSPACE_TOKENS 16

/* Bytes of workspace linear_w8a8_fwd needs for these operands: an f16 copy of
 * int8 weights when there are many tokens, and copies at a 16-byte pitch of
 * rows that are not 16-byte aligned (base and stride).  Host-only. */
size_t linear_w8a8_workspace_size(const void* x, int64_t x_stride, const void* w,
                                  int64_t w_stride, int dtype, int64_t tokens, int64_t outputs,
                                  int64_t width);

#ifdef __cplusplus
}
#endif

#endif /* TOKEN_OPS_GB300_H */
