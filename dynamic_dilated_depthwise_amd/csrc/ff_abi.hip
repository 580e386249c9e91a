// ff_abi.hip -- the exported C ABI of the feed-forward operators (include/ddpm_ff.h): argument
// validation and dispatch.  Validation completes before anything is enqueued.
#include <stdint.h>

#include <algorithm>

#include "abi_check.hpp"
#include "ff_launch.hpp"
#include "ff_plan.hpp"

namespace {

using namespace ddpm::abi;
using namespace ddpm::ff;

bool sizes_ok(Check &c, const Sizes &s, int activation) {
    for (int64_t v : {s.rows, s.C, s.N}) c.size(v, kMaxRun);
    c.bad |= activation < DDPM_ACT_NONE || activation > DDPM_ACT_GELU;
    return !c.bad && (double)s.rows * s.width <= kMostElements && (double)s.rows * s.C <= kMostElements &&
           (double)s.width * s.C <= kMostElements;
}

// Copies x and weight to `work` and points the product at them.
hipError_t copy_operands(const Sizes &s, const void *&x, int64_t &x_row, const void *&weight, int64_t &weight_row, char *&work,
                         bool bf16, hipStream_t stream) {
    const Copy cx = {x, x_row, s.rows, s.C, work}, cw = {weight, s.C, s.width, s.C, work + x_copy_bytes(s, bf16)};
    x = cx.dst;
    weight = cw.dst;
    x_row = weight_row = padded(s.C, bf16);
    work += x_copy_bytes(s, bf16) + weight_copy_bytes(s, bf16);
    return launch_copies(cx, cw, bf16, stream);
}

int64_t forward_workspace(Kind kind, const Sizes &s, int dtype) {
    Check c(dtype);
    if (!sizes_ok(c, s, DDPM_ACT_NONE)) return 0;
    const bool bf16 = is_bf16(dtype);
    return (forward_copies(kind, s, bf16) ? x_copy_bytes(s, bf16) + weight_copy_bytes(s, bf16) : 0) +
           product_bytes(kind, s.N, s.rows, s.C, 1, bf16);
}

int64_t saved_count(const Sizes &s, bool gated, int activation, int dtype) {
    Check c(dtype);
    return sizes_ok(c, s, activation) ? saved_floats(s, gated || activation != DDPM_ACT_NONE, is_bf16(dtype)) : 0;
}

int forward(Kind kind, const void *x, const void *weight, const void *bias, const void *residual, void *y, float *saved,
            void *workspace, const Sizes &s, int64_t x_row, int64_t residual_row, int activation, int dtype,
            hipStream_t stream) {
    Check c(dtype);
    if (!sizes_ok(c, s, activation)) return DDPM_ERR_INVALID_ARG;
    c.stride(x_row);
    if (residual != nullptr) c.stride(residual_row);
    if (c.bad) return DDPM_ERR_INVALID_ARG;
    const bool bf16 = is_bf16(dtype), through = kind == kGatedForward || activation != DDPM_ACT_NONE;
    c.input(x, extent(1, s.rows, s.C, 0, x_row), c.es());
    c.input(weight, (double)s.width * s.C, c.es());
    c.maybe_in(bias, s.width, c.es());
    if (residual != nullptr) c.input(residual, extent(1, s.rows, s.N, 0, residual_row), c.es());
    c.output(y, (double)s.rows * s.N, c.es());
    if (!through && saved != nullptr) return DDPM_ERR_INVALID_ARG;
    c.maybe_out(saved, (double)saved_floats(s, through, bf16), 4);
    const int64_t room = forward_workspace(kind, s, dtype);
    if (room > 0) c.workspace(workspace, (double)room);
    const int st = c.done();
    if (st != DDPM_OK) return st;
    (void)hipGetLastError();
    char *work = (char *)workspace;
    int64_t weight_row = s.C;
    Product a = {};
    if (forward_copies(kind, s, bf16)) {
        const hipError_t e = copy_operands(s, x, x_row, weight, weight_row, work, bf16, stream);
        if (e != hipSuccess) return status_of(e);
        a.p_padded = a.q_padded = true;
    }
    a.p = weight;
    a.q = x;
    a.p_ld = weight_row;
    a.q_ld = x_row;
    a.np = s.N;
    a.nq = s.rows;
    a.nk = s.C;
    a.out = y;
    (makes_again(s, bf16) ? a.kept : a.saved) = saved;
    a.bias = bias;
    a.residual = residual;
    a.residual_ld = residual_row;
    a.act = activation;
    return status_of(launch_product(kind, a, work, bf16, stream));
}

int64_t backward_workspace(Kind kind, const Sizes &s, bool through, int activation, int dtype) {
    Check c(dtype);
    return sizes_ok(c, s, activation) ? backward_room(kind, s, through, activation, is_bf16(dtype)).all : 0;
}

int backward(Kind kind, const void *grad, const void *x, const void *weight, const float *saved, void *grad_x,
             void *grad_weight, void *grad_bias, void *workspace, const Sizes &s, int64_t x_row, int64_t grad_row,
             int activation, int dtype, hipStream_t stream) {
    Check c(dtype);
    if (!sizes_ok(c, s, activation) || (grad_weight == nullptr) != (grad_bias == nullptr)) return DDPM_ERR_INVALID_ARG;
    c.stride(x_row);
    c.stride(grad_row);
    if (c.bad) return DDPM_ERR_INVALID_ARG;
    const bool gated = kind == kGatedForward, through = gated || activation != DDPM_ACT_NONE, bf16 = is_bf16(dtype);
    c.input(grad, extent(1, s.rows, s.N, 0, grad_row), c.es());
    c.input(x, extent(1, s.rows, s.C, 0, x_row), c.es());
    c.input(weight, (double)s.width * s.C, c.es());
    if (through) c.input(saved, (double)saved_floats(s, through, bf16), 4);
    c.maybe_out(grad_x, (double)s.rows * s.C, c.es());
    c.maybe_out(grad_weight, (double)s.width * s.C, c.es());
    c.maybe_out(grad_bias, s.width, c.es());
    const Room room = backward_room(kind, s, through, activation, bf16);
    if (room.all > 0) c.workspace(workspace, (double)room.all);
    const int st = c.done();
    if (st != DDPM_OK) return st;
    (void)hipGetLastError();
    if (room.small) {
        const SmallBackward b = {grad, x, weight, saved, s.rows, grad_row, x_row, s.C, (int)s.C, (int)s.N, activation, grad_x,
                                 grad_weight != nullptr ? (float *)workspace : nullptr};
        return status_of(launch_small_backward(gated, b, grad_weight, grad_bias, bf16, stream));
    }
    char *work = (char *)workspace + room.dz;
    int64_t weight_row = s.C;
    hipError_t e = hipSuccess;
    if (room.copies) e = copy_operands(s, x, x_row, weight, weight_row, work, bf16, stream);
    if (e == hipSuccess && room.own_dz) {
        if (room.again) {
            Product z = {};
            z.p = weight;
            z.q = x;
            z.p_ld = weight_row;
            z.q_ld = x_row;
            z.p_padded = z.q_padded = room.copies;
            z.np = s.N;
            z.nq = s.rows;
            z.nk = s.C;
            z.out = workspace;
            z.low = room.low;
            z.kept = const_cast<float *>(saved);
            z.grad = grad;
            z.grad_ld = grad_row;
            z.act = activation;
            e = launch_product(kind, z, work, bf16, stream);
        } else if (through) {
            e = launch_dz(gated, grad, grad_row, saved, workspace, room.low, s.rows, s.N, activation, bf16, stream);
        } else {
            e = launch_copies({grad, grad_row, s.rows, s.N, workspace}, {}, bf16, stream);
        }
    }
    Product a = {};
    a.q = room.own_dz ? workspace : grad;
    a.q_ld = room.own_dz ? padded(s.width, bf16) : grad_row;
    a.q_padded = room.own_dz;
    a.low = room.low;
    a.p_padded = room.copies;
    a.np = s.C;
    if (e == hipSuccess && grad_x != nullptr) {
        Product b = a;
        b.p = weight;
        b.p_ld = weight_row;
        b.nq = s.rows;
        b.nk = s.width;
        b.out = grad_x;
        e = launch_product(kGradX, b, work, bf16, stream);
    }
    if (e == hipSuccess && grad_weight != nullptr) {
        a.p = x;
        a.p_ld = x_row;
        a.nq = s.width;
        a.nk = s.rows;
        a.out = grad_weight;
        a.sums = grad_bias;
        e = launch_product(kGradWeight, a, work, bf16, stream);
    }
    return status_of(e);
}

}  // namespace

extern "C" {

int64_t ddpm_linear_fwd_workspace(int64_t rows, int64_t C, int64_t N, int dtype) {
    return forward_workspace(kForward, {rows, C, N, N}, dtype);
}

int ddpm_linear_fwd(const void *x, const void *weight, const void *bias, const void *residual, void *y, float *saved,
                    void *workspace, int64_t rows, int64_t C, int64_t N, int64_t x_row, int64_t residual_row,
                    int activation, int dtype, hipStream_t stream) {
    return forward(kForward, x, weight, bias, residual, y, saved, workspace, {rows, C, N, N}, x_row, residual_row, activation,
                   dtype, stream);
}

int64_t ddpm_linear_saved(int64_t rows, int64_t C, int64_t N, int activation, int dtype) {
    return saved_count({rows, C, N, N}, false, activation, dtype);
}

int64_t ddpm_linear_bwd_workspace(int64_t rows, int64_t C, int64_t N, int activation, int dtype) {
    return backward_workspace(kForward, {rows, C, N, N}, activation != DDPM_ACT_NONE, activation, dtype);
}

int ddpm_linear_bwd(const void *grad, const void *x, const void *weight, const float *saved, void *grad_x,
                    void *grad_weight, void *grad_bias, void *workspace, int64_t rows, int64_t C, int64_t N, int64_t x_row,
                    int64_t grad_row, int activation, int dtype, hipStream_t stream) {
    return backward(kForward, grad, x, weight, saved, grad_x, grad_weight, grad_bias, workspace, {rows, C, N, N}, x_row, grad_row,
                    activation, dtype, stream);
}

int64_t ddpm_gated_linear_fwd_workspace(int64_t rows, int64_t C, int64_t N, int dtype) {
    return forward_workspace(kGatedForward, {rows, C, N, 2 * N}, dtype);
}

int ddpm_gated_linear_fwd(const void *x, const void *weight, const void *bias, void *y, float *saved, void *workspace,
                          int64_t rows, int64_t C, int64_t N, int64_t x_row, int activation, int dtype, hipStream_t stream) {
    return forward(kGatedForward, x, weight, bias, nullptr, y, saved, workspace, {rows, C, N, 2 * N}, x_row, 0, activation, dtype,
                   stream);
}

int64_t ddpm_gated_linear_saved(int64_t rows, int64_t C, int64_t N, int dtype) {
    return saved_count({rows, C, N, 2 * N}, true, DDPM_ACT_NONE, dtype);
}

int64_t ddpm_gated_linear_bwd_workspace(int64_t rows, int64_t C, int64_t N, int dtype) {
    return backward_workspace(kGatedForward, {rows, C, N, 2 * N}, true, DDPM_ACT_NONE, dtype);
}

int ddpm_gated_linear_bwd(const void *grad, const void *x, const void *weight, const float *saved, void *grad_x,
                          void *grad_weight, void *grad_bias, void *workspace, int64_t rows, int64_t C, int64_t N,
                          int64_t x_row, int64_t grad_row, int activation, int dtype, hipStream_t stream) {
    return backward(kGatedForward, grad, x, weight, saved, grad_x, grad_weight, grad_bias, workspace, {rows, C, N, 2 * N}, x_row, grad_row,
                    activation, dtype, stream);
}

}  // extern "C"
