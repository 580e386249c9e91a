// seq_abi.hip -- the exported C ABI of the sequence operators (include/ddpm_seq.h):
// argument validation and dispatch.  Validation completes before anything is enqueued.
#include <stdint.h>

#include "../../include/ddpm_seq.h"
#include "abi_check.hpp"
#include "seq_launch.hpp"

namespace {

using namespace ddpm::abi;

int conv_sizes(Check &c, int64_t batch, int64_t length, int64_t D, int width, int64_t x_batch, int64_t x_token) {
    c.size(batch);
    c.size(length, kMaxRun);
    c.size(D, kMaxRun);
    c.size(width);
    c.stride(x_batch);
    c.stride(x_token);
    if (c.bad || (double)batch * length * D > kMostElements) return DDPM_ERR_INVALID_ARG;
    return width > DDPM_SEQ_MAX_WIDTH ? DDPM_ERR_UNSUPPORTED : DDPM_OK;
}

bool scan_sizes_ok(const ddpm_scan *s) {
    if (s == nullptr || (s->dtype != DDPM_F32 && s->dtype != DDPM_BF16)) return false;
    for (int64_t v : {s->batch, s->length, (int64_t)s->heads, (int64_t)s->P, (int64_t)s->groups, (int64_t)s->N})
        if (v < 1 || v > kMax) return false;
    // a head's state, its rows padded, and a token's rows are walked as ints
    if (s->length > kMaxRun || (int64_t)s->P * (s->N + 3) > kMaxRun || (int64_t)s->heads * s->P > kMaxRun ||
        (int64_t)s->groups * s->N > kMaxRun)
        return false;
    const double tokens = (double)s->batch * (s->length + 1024);
    if (tokens * s->heads * s->P > kMostElements || tokens * s->groups * s->N > kMostElements ||
        tokens / 64 * s->heads * s->P * s->N > kMostElements)
        return false;
    return s->heads % s->groups == 0;
}

// What the scan's calls share.
void scan_inputs(Check &c, const ddpm_scan *s, int64_t length) {
    for (int64_t v : {s->x_batch, s->x_token, s->dt_batch, s->dt_token, s->B_batch, s->B_token, s->C_batch, s->C_token})
        c.stride(v);
    if (c.bad) return;
    const int64_t gn = (int64_t)s->groups * s->N, es = c.es();
    c.input(s->x, extent(s->batch, length, (int64_t)s->heads * s->P, s->x_batch, s->x_token), es);
    c.input(s->dt, extent(s->batch, length, s->heads, s->dt_batch, s->dt_token), es);
    c.input(s->B, extent(s->batch, length, gn, s->B_batch, s->B_token), es);
    c.input(s->C, extent(s->batch, length, gn, s->C_batch, s->C_token), es);
    c.input(s->A, s->heads, 4);
    c.input(s->D, s->heads, 4);
    c.input(s->dt_bias, s->heads, 4);
}

ddpm::seq::Scan scan_of(const ddpm_scan *s) {
    return {s->x, s->dt, s->B, s->C, s->A, s->D, s->dt_bias, s->initial_state, s->lengths, s->x_batch, s->x_token,
            s->dt_batch, s->dt_token, s->B_batch, s->B_token, s->C_batch, s->C_token, s->batch, s->length, s->heads, s->P,
            s->groups, s->N};
}

double state_count(const ddpm_scan *s) { return (double)s->batch * s->heads * s->P * s->N; }

}  // namespace

extern "C" {

int ddpm_layer_norm_fwd(const void *x, const void *weight, const void *bias, void *y, float *mean, float *rstd,
                        int64_t rows, int64_t C, int64_t x_row, float eps, int dtype, hipStream_t stream) {
    Check c(dtype);
    c.size(rows);
    c.size(C, kMaxRun);
    c.stride(x_row);
    if (c.bad || !(eps >= 0.f) || (mean == nullptr) != (rstd == nullptr)) return DDPM_ERR_INVALID_ARG;
    c.input(x, extent(1, rows, C, 0, x_row), c.es());
    c.input(weight, C, c.es());
    c.input(bias, C, c.es());
    c.output(y, (double)rows * C, c.es());
    c.maybe_out(mean, rows, 4);
    c.maybe_out(rstd, rows, 4);
    const int st = c.done();
    if (st != DDPM_OK) return st;
    (void)hipGetLastError();
    return status_of(ddpm::seq::launch_norm_fwd(x, weight, bias, y, mean, rstd, rows, C, x_row, eps, is_bf16(dtype), stream));
}

int64_t ddpm_layer_norm_bwd_workspace(int64_t rows, int64_t C, int dtype) {
    Check c(dtype);
    c.size(rows);
    c.size(C, kMaxRun);
    return c.bad ? 0 : (int64_t)ddpm::seq::norm_partials(rows, C, is_bf16(dtype)) * 2 * C * 4;
}

int ddpm_layer_norm_bwd(const void *grad, const void *x, const void *weight, const float *mean, const float *rstd,
                        void *grad_x, void *grad_weight, void *grad_bias, void *workspace, int64_t rows, int64_t C,
                        int64_t x_row, int64_t grad_row, int dtype, hipStream_t stream) {
    Check c(dtype);
    c.size(rows);
    c.size(C, kMaxRun);
    c.stride(x_row);
    c.stride(grad_row);
    if (c.bad) return DDPM_ERR_INVALID_ARG;
    c.input(grad, extent(1, rows, C, 0, grad_row), c.es());
    c.input(x, extent(1, rows, C, 0, x_row), c.es());
    c.input(weight, C, c.es());
    c.input(mean, rows, 4);
    c.input(rstd, rows, 4);
    c.output(grad_x, (double)rows * C, c.es());
    c.output(grad_weight, C, c.es());
    c.output(grad_bias, C, c.es());
    c.workspace(workspace, (double)ddpm_layer_norm_bwd_workspace(rows, C, dtype));
    const int st = c.done();
    if (st != DDPM_OK) return st;
    (void)hipGetLastError();
    return status_of(ddpm::seq::launch_norm_bwd(grad, x, weight, mean, rstd, grad_x, grad_weight, grad_bias,
                                                (float *)workspace, rows, C, x_row, grad_row, is_bf16(dtype), stream));
}

int ddpm_causal_conv_fwd(const void *x, const void *weight, const void *bias, const void *initial_state,
                         const int32_t *lengths, void *y, void *final_state, int64_t batch, int64_t length, int64_t D,
                         int width, int64_t x_batch, int64_t x_token, int dtype, hipStream_t stream) {
    Check c(dtype);
    int st = conv_sizes(c, batch, length, D, width, x_batch, x_token);
    if (st != DDPM_OK) return st;
    const double state = (double)batch * (width - 1) * D;
    if (width == 1 && (initial_state != nullptr || final_state != nullptr)) return DDPM_ERR_INVALID_ARG;
    c.input(x, extent(batch, length, D, x_batch, x_token), c.es());
    c.input(weight, (double)D * width, c.es());
    c.input(bias, D, c.es());
    c.maybe_in(initial_state, state, c.es());
    c.maybe_in(lengths, batch, 4);
    c.output(y, (double)batch * length * D, c.es());
    c.maybe_out(final_state, state, c.es());
    st = c.done();
    if (st != DDPM_OK) return st;
    const ddpm::seq::Conv a = {x, weight, bias, initial_state, lengths, batch, length, D, x_batch, x_token, width};
    (void)hipGetLastError();
    return status_of(ddpm::seq::launch_conv_fwd(a, y, final_state, is_bf16(dtype), stream));
}

int64_t ddpm_causal_conv_bwd_workspace(int64_t batch, int64_t length, int64_t D, int width, int dtype) {
    Check c(dtype);
    if (conv_sizes(c, batch, length, D, width, 0, 0) != DDPM_OK) return 0;
    return (int64_t)ddpm::seq::conv_partials(batch, length, D, width) * D * (width + 1) * 4;
}

int ddpm_causal_conv_bwd(const void *grad, const void *x, const void *weight, const void *bias,
                         const void *initial_state, const int32_t *lengths, const void *grad_state, void *grad_x,
                         void *grad_weight, void *grad_bias, void *grad_initial, void *workspace, int64_t batch,
                         int64_t length, int64_t D, int width, int64_t x_batch, int64_t x_token, int64_t grad_batch,
                         int64_t grad_token, int dtype, hipStream_t stream) {
    Check c(dtype);
    c.stride(grad_batch);
    c.stride(grad_token);
    int st = conv_sizes(c, batch, length, D, width, x_batch, x_token);
    if (st != DDPM_OK) return st;
    const double state = (double)batch * (width - 1) * D;
    if (width == 1 && (initial_state != nullptr || grad_state != nullptr || grad_initial != nullptr))
        return DDPM_ERR_INVALID_ARG;
    c.input(grad, extent(batch, length, D, grad_batch, grad_token), c.es());
    c.input(x, extent(batch, length, D, x_batch, x_token), c.es());
    c.input(weight, (double)D * width, c.es());
    c.input(bias, D, c.es());
    c.maybe_in(initial_state, state, c.es());
    c.maybe_in(lengths, batch, 4);
    c.maybe_in(grad_state, state, c.es());
    c.output(grad_x, (double)batch * length * D, c.es());
    c.output(grad_weight, (double)D * width, c.es());
    c.output(grad_bias, D, c.es());
    c.maybe_out(grad_initial, state, c.es());
    c.workspace(workspace, (double)ddpm_causal_conv_bwd_workspace(batch, length, D, width, dtype));
    st = c.done();
    if (st != DDPM_OK) return st;
    const ddpm::seq::Conv a = {x, weight, bias, initial_state, lengths, batch, length, D, x_batch, x_token, width};
    (void)hipGetLastError();
    return status_of(ddpm::seq::launch_conv_bwd(a, grad, grad_batch, grad_token, grad_state, grad_x, grad_initial,
                                                grad_weight, grad_bias, (float *)workspace, is_bf16(dtype), stream));
}

int ddpm_causal_conv_step(const void *x, const void *weight, const void *bias, void *state, const int32_t *slots,
                          void *y, int64_t batch, int64_t num_slots, int64_t D, int width, int64_t x_batch, int dtype,
                          hipStream_t stream) {
    Check c(dtype);
    c.size(num_slots);
    int st = conv_sizes(c, batch, 1, D, width, x_batch, 0);
    if (st != DDPM_OK) return st;
    if (slots == nullptr && num_slots < batch) return DDPM_ERR_INVALID_ARG;
    c.input(x, extent(batch, 1, D, x_batch, 0), c.es());
    c.input(weight, (double)D * width, c.es());
    c.input(bias, D, c.es());
    c.maybe_in(slots, batch, 4);
    c.output(y, (double)batch * D, c.es());
    if (width > 1) c.output(state, (double)num_slots * (width - 1) * D, c.es());
    else if (state != nullptr) return DDPM_ERR_INVALID_ARG;
    st = c.done();
    if (st != DDPM_OK) return st;
    (void)hipGetLastError();
    return status_of(ddpm::seq::launch_conv_step(x, x_batch, weight, bias, state, slots, y, batch, num_slots, D, width,
                                                 is_bf16(dtype), stream));
}

int64_t ddpm_selective_scan_fwd_workspace(const ddpm_scan *s) {
    if (!scan_sizes_ok(s)) return 0;
    return 4 * ddpm::seq::scan_fwd_floats(s->batch, s->length, s->heads, s->P, s->groups, s->N, is_bf16(s->dtype));
}

int64_t ddpm_selective_scan_bwd_workspace(const ddpm_scan *s) {
    if (!scan_sizes_ok(s)) return 0;
    return 4 * ddpm::seq::scan_bwd_floats(s->batch, s->length, s->heads, s->P, s->groups, s->N, is_bf16(s->dtype));
}

int ddpm_selective_scan_fwd(const ddpm_scan *s, void *y, float *final_state, int save, void *workspace,
                            hipStream_t stream) {
    if (!scan_sizes_ok(s)) return DDPM_ERR_INVALID_ARG;
    if (s->N > DDPM_SEQ_MAX_STATE) return DDPM_ERR_UNSUPPORTED;
    Check c(s->dtype);
    scan_inputs(c, s, s->length);
    if (c.bad) return DDPM_ERR_INVALID_ARG;
    c.maybe_in(s->initial_state, state_count(s), 4);
    c.maybe_in(s->lengths, s->batch, 4);
    c.output(y, (double)s->batch * s->length * s->heads * s->P, c.es());
    c.maybe_out(final_state, state_count(s), 4);
    c.workspace(workspace, (double)ddpm_selective_scan_fwd_workspace(s));
    const int st = c.done();
    if (st != DDPM_OK) return st;
    (void)hipGetLastError();
    return status_of(ddpm::seq::launch_scan_fwd(scan_of(s), (float *)workspace, y, final_state, save != 0,
                                                is_bf16(s->dtype), stream));
}

int ddpm_selective_scan_bwd(const ddpm_scan *s, const void *saved, const void *grad, int64_t grad_batch,
                            int64_t grad_token, const float *grad_state, void *grad_x, void *grad_dt, float *grad_A,
                            void *grad_B, void *grad_C, float *grad_D, float *grad_dt_bias, float *grad_initial,
                            void *workspace, hipStream_t stream) {
    if (!scan_sizes_ok(s)) return DDPM_ERR_INVALID_ARG;
    if (s->N > DDPM_SEQ_MAX_STATE) return DDPM_ERR_UNSUPPORTED;
    Check c(s->dtype);
    c.stride(grad_batch);
    c.stride(grad_token);
    scan_inputs(c, s, s->length);
    if (c.bad) return DDPM_ERR_INVALID_ARG;
    const double tokens = (double)s->batch * s->length, xs = tokens * s->heads * s->P, bs = tokens * s->groups * s->N;
    c.maybe_in(s->initial_state, state_count(s), 4);
    c.maybe_in(s->lengths, s->batch, 4);
    c.input(grad, extent(s->batch, s->length, (int64_t)s->heads * s->P, grad_batch, grad_token), c.es());
    c.maybe_in(grad_state, state_count(s), 4);
    c.pointer(saved, 16);
    c.input(saved, (double)ddpm_selective_scan_fwd_workspace(s) / 4, 4);
    c.output(grad_x, xs, c.es());
    c.output(grad_dt, tokens * s->heads, c.es());
    c.output(grad_A, s->heads, 4);
    c.output(grad_B, bs, c.es());
    c.output(grad_C, bs, c.es());
    c.output(grad_D, s->heads, 4);
    c.output(grad_dt_bias, s->heads, 4);
    c.maybe_out(grad_initial, state_count(s), 4);
    c.workspace(workspace, (double)ddpm_selective_scan_bwd_workspace(s));
    const int st = c.done();
    if (st != DDPM_OK) return st;
    (void)hipGetLastError();
    return status_of(ddpm::seq::launch_scan_bwd(scan_of(s), (const float *)saved, grad, grad_batch, grad_token, grad_state,
                                                (float *)workspace, grad_x, grad_dt, grad_A, grad_B, grad_C, grad_D,
                                                grad_dt_bias, grad_initial, is_bf16(s->dtype), stream));
}

int ddpm_selective_scan_step(const ddpm_scan *s, float *state, const int32_t *slots, int64_t num_slots, void *y,
                             hipStream_t stream) {
    if (!scan_sizes_ok(s) || s->length != 1 || num_slots < 1 || num_slots > kMax) return DDPM_ERR_INVALID_ARG;
    if (slots == nullptr && num_slots < s->batch) return DDPM_ERR_INVALID_ARG;
    Check c(s->dtype);
    scan_inputs(c, s, 1);
    if (c.bad) return DDPM_ERR_INVALID_ARG;
    c.maybe_in(slots, s->batch, 4);
    c.output(y, (double)s->batch * s->heads * s->P, c.es());
    c.output(state, (double)num_slots * s->heads * s->P * s->N, 4);
    const int st = c.done();
    if (st != DDPM_OK) return st;
    (void)hipGetLastError();
    return status_of(ddpm::seq::launch_scan_step(scan_of(s), state, slots, num_slots, y, is_bf16(s->dtype), stream));
}

}  // extern "C"
