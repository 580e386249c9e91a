/*
 * ddpm_ff.h -- C ABI of the feed-forward operators: a matrix product with bias, activation and
 * residual in its epilogue and the gated projection of a feed-forward block, forward and
 * backward.  The same library (libddpm.so), status codes and dtypes as ddpm.h.
 *
 * Conventions
 * -----------
 * Memory.  Every pointer is a DEVICE pointer owned by the caller.  x, residual and grad may be
 *   views whose last axis is contiguous, `*_row` is the stride of their rows in elements, not
 *   negative.  Everything else, and every output, is contiguous.  Pointers are aligned to their
 *   element.  Outputs must not overlap inputs or each other.  The library allocates nothing:
 *   workspaces come from the caller, 16-byte aligned, of the size that the matching *_workspace
 *   function returns in bytes (NULL where that is 0; their contents need no preparation).
 * Alignment costs time only.  Products are fastest where the rows of x, weight and grad start at
 *   multiples of 16 bytes.  Rows of C elements that are no such multiple are copied where that pays;
 *   views whose address or stride is none are not, and take 1.3 to 3 times as long (4096^3, us: y, grad_x
 *   and grad_weight in bfloat16 113, 112, 114, from odd addresses 174, 180, 371; in float32 603, 608,
 *   611, and 794, 829, 839).
 * Streams.  As in ddpm.h: work is enqueued on `stream` and the call returns.  Nothing is cleared
 *   by memset, so every call may be captured into a graph.  No atomics are used: equal inputs
 *   at equally aligned addresses give equal bits.
 * Precision.  Products are summed in float32; float32 operands enter the matrix instructions as
 *   three bfloat16 terms each, six products of them, which is float32's own precision (operands
 *   below 2^-110 lose bits of the third term, at 2^-126 all but eight); up to 64 rows of a forward
 *   whose rows are no whole 16-byte chunks may be multiplied in float32 itself.  Bias,
 *   activation and residual are applied to that sum, and outputs are rounded once.  In the
 *   backward of an activation or a gate the gradient of its input enters the two products in
 *   float32 or as two bfloat16 terms.
 * Not finite.  An infinity or NaN in a row of x or grad reaches that row of y or grad_x, and the
 *   parameters' gradients, and no other row.  In float32 an infinity in an operand of a product may
 *   give NaN where the sum is infinite; finite operands give what float32 holds of their sum, up to
 *   the largest of them (a sum that leaves float32's range gives an infinity or NaN).
 * Errors.  As in ddpm.h; all arguments are checked before anything is enqueued.
 *     DDPM_ERR_INVALID_ARG  null or misaligned pointers, sizes below 1 or beyond 2^31 - 2^16,
 *                           negative strides, an unknown dtype or activation, overlapping
 *                           outputs, one of grad_weight and grad_bias without the other;
 *     DDPM_ERR_UNSUPPORTED  a grid beyond 2^31 - 1 workgroups.
 */
#ifndef DDPM_FF_H_
#define DDPM_FF_H_

#include "ddpm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* none: z; relu: max(z, 0); silu: z / (1 + exp(-z)); gelu: z Phi(z), Phi the normal distribution */
typedef enum { DDPM_ACT_NONE = 0, DDPM_ACT_RELU = 1, DDPM_ACT_SILU = 2, DDPM_ACT_GELU = 3 } ddpm_activation;

/*
 * z = x weight^T + bias,  y = act(z) + residual:  x [rows, C], weight [N, C], bias [N] or NULL,
 * residual [rows, N] or NULL, y [rows, N].  saved, or NULL, receives what the backward of an
 * activation takes: *_saved floats (z, or where making z again costs less, the bias; none, and
 * NULL, with DDPM_ACT_NONE).
 */
int64_t ddpm_linear_saved(int64_t rows, int64_t C, int64_t N, int activation, int dtype);
int64_t ddpm_linear_fwd_workspace(int64_t rows, int64_t C, int64_t N, int dtype);
int ddpm_linear_fwd(const void *x, const void *weight, const void *bias, const void *residual, void *y, float *saved,
                    void *workspace, int64_t rows, int64_t C, int64_t N, int64_t x_row, int64_t residual_row,
                    int activation, int dtype, hipStream_t stream);
/*
 * dz = grad act'(z),  grad_x = dz weight,  grad_weight = dz^T x,  grad_bias = sums of dz over the
 * rows; the residual's gradient is grad.  saved is the forward's (NULL with DDPM_ACT_NONE).
 * grad_x may be NULL, and grad_weight with grad_bias.
 */
int64_t ddpm_linear_bwd_workspace(int64_t rows, int64_t C, int64_t N, int activation, int dtype);
int ddpm_linear_bwd(const void *grad, const void *x, const void *weight, const float *saved, void *grad_x,
                    void *grad_weight, void *grad_bias, void *workspace, int64_t rows, int64_t C, int64_t N, int64_t x_row,
                    int64_t grad_row, int activation, int dtype, hipStream_t stream);

/*
 * [g, u] = x weight^T + bias, N columns each,  y = act(g) u:  x [rows, C], weight [2 N, C] (g's
 * rows, then u's), bias [2 N] or NULL, y [rows, N].  saved, or NULL, receives what the backward
 * takes: *_saved floats.
 */
int64_t ddpm_gated_linear_saved(int64_t rows, int64_t C, int64_t N, int dtype);
int64_t ddpm_gated_linear_fwd_workspace(int64_t rows, int64_t C, int64_t N, int dtype);
int ddpm_gated_linear_fwd(const void *x, const void *weight, const void *bias, void *y, float *saved, void *workspace,
                          int64_t rows, int64_t C, int64_t N, int64_t x_row, int activation, int dtype, hipStream_t stream);
/*
 * dg = grad u act'(g), du = grad act(g);  with dz = [dg, du]: grad_x = dz weight,
 * grad_weight = dz^T x, grad_bias = sums of dz over the rows.  grad_x may be NULL, and
 * grad_weight with grad_bias.
 */
int64_t ddpm_gated_linear_bwd_workspace(int64_t rows, int64_t C, int64_t N, int dtype);
int ddpm_gated_linear_bwd(const void *grad, const void *x, const void *weight, const float *saved, void *grad_x,
                          void *grad_weight, void *grad_bias, void *workspace, int64_t rows, int64_t C, int64_t N,
                          int64_t x_row, int64_t grad_row, int activation, int dtype, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DDPM_FF_H_ */
