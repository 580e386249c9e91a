/*
 * ddpm_seq.h -- C ABI of the sequence operators: layer norm, short causal convolution and
 * selective state space scan, forward and backward over whole sequences and one token at a
 * time.  The same library (libddpm.so), status codes and dtypes as ddpm.h.
 *
 * Conventions
 * -----------
 * Memory.  Every pointer is a DEVICE pointer owned by the caller.  Inputs named with a
 *   stride may be views: the last axis (of x, B and C of the scan the last two) is
 *   contiguous, `*_batch` and `*_token` are the strides, in elements and not negative, of
 *   the two axes before it.  Everything else, and every output, is contiguous.  Pointers
 *   are aligned to their element.  Outputs must not overlap inputs or each other, except
 *   the states that the step functions update in place.  The library allocates nothing:
 *   workspaces come from the caller, 16-byte aligned, of the size that the matching
 *   *_workspace function returns in bytes (their contents need no preparation).
 * Streams.  As in ddpm.h: work is enqueued on `stream` and the call returns.  Nothing is
 *   cleared by memset, so every call may be captured into a graph.  No atomics are used:
 *   equal inputs give equal bits.
 * Precision.  All sums, statistics, decays and states are float32 or wider.  bfloat16
 *   outputs are rounded once, from float32; matrix operands made on the way are two bfloat16
 *   terms (17 bits) where the type is bfloat16, and where they lead to float32 outputs (final
 *   state, grad_A, grad_D, grad_dt_bias) or grad_dt three or more.
 * Lengths.  `lengths` [batch] int32, or NULL: sequence b has lengths[b] tokens (values
 *   outside [0, length] are taken as the nearest).  Later positions are not read; y and the
 *   gradients there are zero and the state is that behind the last token.
 * Not finite.  In the scan an infinity or NaN of a token reaches y of that token and later ones
 *   and the states, as in the recurrence, and nothing before it.  In its backward any gradient of
 *   the same chunk of tokens (128 in bfloat16, 64 in float32) and head or group may become NaN.
 * Slots.  `slots` [batch] int32, or NULL for 0, 1, ...: the state of sequence b is
 *   state[slots[b]].  A slot outside [0, num_slots) marks a place without a sequence: y is
 *   zero and no state is touched.  A slot may be named once in a call.  Without slots
 *   num_slots is at least batch.
 * Errors.  As in ddpm.h; all arguments are checked before anything is enqueued.
 *     DDPM_ERR_INVALID_ARG  null or misaligned pointers, sizes below 1 or beyond 2^31 - 1
 *                           (2^31 - 2^16 for C, length and D, and in the scan for heads * P,
 *                           groups * N and P * (N + 3)), a negative or NaN eps, negative
 *                           strides, an unknown dtype, overlapping outputs, heads not a
 *                           multiple of groups;
 *     DDPM_ERR_UNSUPPORTED  width > 8, state columns N > 128 (scan over sequences), or a
 *                           grid beyond 2^31 - 1 workgroups.
 */
#ifndef DDPM_SEQ_H_
#define DDPM_SEQ_H_

#include "ddpm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DDPM_SEQ_MAX_WIDTH 8
#define DDPM_SEQ_MAX_STATE 128

/*
 * Layer norm over the last axis of [rows, C]:
 *   y = (x - mean) * rstd * weight + bias,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
 * x has row stride x_row.  mean and rstd [rows] float32 are both written or both NULL; the
 * backward takes them.
 */
int ddpm_layer_norm_fwd(const void *x, const void *weight, const void *bias, void *y, float *mean, float *rstd,
                        int64_t rows, int64_t C, int64_t x_row, float eps, int dtype, hipStream_t stream);
int64_t ddpm_layer_norm_bwd_workspace(int64_t rows, int64_t C, int dtype);
int ddpm_layer_norm_bwd(const void *grad, const void *x, const void *weight, const float *mean, const float *rstd,
                        void *grad_x, void *grad_weight, void *grad_bias, void *workspace, int64_t rows, int64_t C,
                        int64_t x_row, int64_t grad_row, int dtype, hipStream_t stream);

/*
 * Causal convolution of each channel along the sequence, then SiLU: x [batch, length, D],
 * weight [D, width], bias [D],
 *   u[t] = bias + sum_j weight[:, j] * x[t - (width - 1) + j],  y = u * sigmoid(u).
 * initial_state [batch, width - 1, D] holds the inputs before the first token (NULL: zeros),
 * final_state the last width - 1 inputs (NULL: not written); with width 1 both are NULL.
 */
int ddpm_causal_conv_fwd(const void *x, const void *weight, const void *bias, const void *initial_state,
                         const int32_t *lengths, void *y, void *final_state, int64_t batch, int64_t length, int64_t D,
                         int width, int64_t x_batch, int64_t x_token, int dtype, hipStream_t stream);
int64_t ddpm_causal_conv_bwd_workspace(int64_t batch, int64_t length, int64_t D, int width, int dtype);
/* grad_state (of final_state) and grad_initial may be NULL. */
int ddpm_causal_conv_bwd(const void *grad, const void *x, const void *weight, const void *bias,
                         const void *initial_state, const int32_t *lengths, const void *grad_state, void *grad_x,
                         void *grad_weight, void *grad_bias, void *grad_initial, void *workspace, int64_t batch,
                         int64_t length, int64_t D, int width, int64_t x_batch, int64_t x_token, int64_t grad_batch,
                         int64_t grad_token, int dtype, hipStream_t stream);
/* One token: x and y [batch, D], state [num_slots, width - 1, D] (NULL with width 1). */
int ddpm_causal_conv_step(const void *x, const void *weight, const void *bias, void *state, const int32_t *slots,
                          void *y, int64_t batch, int64_t num_slots, int64_t D, int width, int64_t x_batch, int dtype,
                          hipStream_t stream);

/*
 * Selective scan.  Head h of group h / (heads / groups) keeps a state [P, N], float32:
 *   dt[t] = softplus(raw[t] + dt_bias),  state = exp(dt[t] A) state + dt[t] x[t] (outer) B[t],
 *   y[t] = state C[t] + D x[t].
 * x [batch, length, heads, P], dt (the raw values) [batch, length, heads], B and C
 * [batch, length, groups, N] in dtype; A, D, dt_bias [heads] and initial_state
 * [batch, heads, P, N] (or NULL) float32.  The step functions use length = 1, *_batch only
 * and ignore initial_state and lengths.
 */
typedef struct {
    const void *x, *dt, *B, *C;
    const float *A, *D, *dt_bias, *initial_state;
    const int32_t *lengths;
    int64_t batch, length;
    int64_t x_batch, x_token, dt_batch, dt_token, B_batch, B_token, C_batch, C_token;
    int32_t heads, P, groups, N, dtype;
} ddpm_scan;

/* The forward's workspace (pointers are not read).  Kept unchanged, with save != 0, it is
 * what the backward calls `saved`: times and the states that enter the chunks. */
int64_t ddpm_selective_scan_fwd_workspace(const ddpm_scan *scan);
/* y [batch, length, heads, P]; final_state [batch, heads, P, N] float32 or NULL. */
int ddpm_selective_scan_fwd(const ddpm_scan *scan, void *y, float *final_state, int save, void *workspace,
                            hipStream_t stream);
int64_t ddpm_selective_scan_bwd_workspace(const ddpm_scan *scan);
/* Gradients in their input's type and shape, contiguous; grad_state (of final_state) and
 * grad_initial float32 or NULL.  initial_state and lengths as in the forward call. */
int ddpm_selective_scan_bwd(const ddpm_scan *scan, const void *saved, const void *grad, int64_t grad_batch,
                            int64_t grad_token, const float *grad_state, void *grad_x, void *grad_dt, float *grad_A,
                            void *grad_B, void *grad_C, float *grad_D, float *grad_dt_bias, float *grad_initial,
                            void *workspace, hipStream_t stream);
/* One token: y [batch, heads, P], state [num_slots, heads, P, N] float32, any N. */
int ddpm_selective_scan_step(const ddpm_scan *scan, float *state, const int32_t *slots, int64_t num_slots, void *y,
                             hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DDPM_SEQ_H_ */
