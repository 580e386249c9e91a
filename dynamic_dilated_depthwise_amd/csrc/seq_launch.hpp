// seq_launch.hpp -- kernel launchers of the sequence operators.  They check nothing but
// grid limits (hipErrorInvalidConfiguration); arguments are validated in seq_abi.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ddpm {
namespace seq {

// out0[m] = sum over s < S of part[s][m] for m < M0, out1 the M1 columns after them.
hipError_t launch_sum_rows(const float *part, int S, int64_t M0, int64_t M1, void *out0, void *out1, bool bf16,
                           hipStream_t stream);

// Rows of the float32 partials [S, 2, C] of launch_norm_bwd.
int norm_partials(int64_t rows, int64_t C, bool bf16);
hipError_t launch_norm_fwd(const void *x, const void *weight, const void *bias, void *y, float *mean, float *rstd,
                           int64_t rows, int64_t C, int64_t x_stride, float eps, bool bf16, hipStream_t stream);
hipError_t launch_norm_bwd(const void *grad, const void *x, const void *weight, const float *mean, const float *rstd,
                           void *grad_x, void *grad_weight, void *grad_bias, float *part, int64_t rows, int64_t C,
                           int64_t x_stride, int64_t g_stride, bool bf16, hipStream_t stream);

// A [B, L, D] tensor whose last axis is contiguous; strides in elements.
struct Conv {
    const void *x, *weight, *bias, *initial;
    const int *lengths;
    int64_t B, L, D, x_batch, x_token;
    int W;
};
// Rows of the float32 partials [S, D * W + D] of launch_conv_bwd.
int conv_partials(int64_t B, int64_t L, int64_t D, int W);
hipError_t launch_conv_fwd(const Conv &a, void *y, void *final_state, bool bf16, hipStream_t stream);
hipError_t launch_conv_bwd(const Conv &a, const void *grad, int64_t g_batch, int64_t g_token, const void *grad_state,
                           void *grad_x, void *grad_initial, void *grad_weight, void *grad_bias, float *part, bool bf16,
                           hipStream_t stream);
hipError_t launch_conv_step(const void *x, int64_t x_stride, const void *weight, const void *bias, void *state,
                            const int *slots, void *y, int64_t B, int64_t S, int64_t D, int W, bool bf16,
                            hipStream_t stream);

// x [B, L, H, P], dt [B, L, H], Bm and Cm [B, L, G, N]; all but the first two axes
// contiguous, strides in elements.  A, D, dt_bias [H] float32.
struct Scan {
    const void *x, *dt, *Bm, *Cm;
    const float *A, *D, *dt_bias, *initial;
    const int *lengths;
    int64_t x_batch, x_token, dt_batch, dt_token, b_batch, b_token, c_batch, c_token;
    int64_t B, L;
    int H, P, G, N;
};

int scan_chunk(bool bf16);
// Floats of the forward's workspace and of the backward's.
int64_t scan_fwd_floats(int64_t B, int64_t L, int H, int P, int G, int N, bool bf16);
int64_t scan_bwd_floats(int64_t B, int64_t L, int H, int P, int G, int N, bool bf16);
hipError_t launch_scan_fwd(const Scan &a, float *work, void *y, float *final_state, bool save, bool bf16,
                           hipStream_t stream);
hipError_t launch_scan_bwd(const Scan &a, const float *saved, const void *grad, int64_t g_batch, int64_t g_token,
                           const float *grad_state, float *work, void *grad_x, void *grad_dt, float *grad_A,
                           void *grad_B, void *grad_C, float *grad_D, float *grad_dt_bias, float *grad_initial,
                           bool bf16, hipStream_t stream);
// One token: x [B, H, P] (row stride), dt [B, H], Bm and Cm [B, G, N], state [S, H, P, N].
hipError_t launch_scan_step(const Scan &a, float *state, const int *slots, int64_t S, void *y, bool bf16,
                            hipStream_t stream);

}  // namespace seq
}  // namespace ddpm
