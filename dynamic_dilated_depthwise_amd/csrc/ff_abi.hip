// ff_abi.hip -- the exported C ABI of the feed-forward operators (include/ddpm_ff.h): argument
// validation and dispatch.  Validation completes before anything is enqueued.
#include <stdint.h>

#include <algorithm>

#include "abi_check.hpp"
#include "ff_launch.hpp"

namespace {

using namespace ddpm::abi;
using namespace ddpm::ff;

// Sizes of a call: x [rows, C], y [rows, N], `width` = N or 2 N columns of z.
struct Sizes {
    int64_t rows, C, N, width;
};

bool sizes_ok(Check &c, const Sizes &s, int activation) {
    for (int64_t v : {s.rows, s.C, s.N}) c.size(v, kMaxRun);
    c.bad |= activation < DDPM_ACT_NONE || activation > DDPM_ACT_GELU;
    return !c.bad && (double)s.rows * s.width <= kMostElements && (double)s.rows * s.C <= kMostElements &&
           (double)s.width * s.C <= kMostElements;
}

int64_t rounded(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// Of the backward: dz, where it is another tensor than grad (behind an activation or a gate, and where
// grad's rows are no whole chunks and many enough), then what the products need.
struct Room {
    int64_t dz, rest;
    int64_t all() const { return dz + rest; }
};
Room backward_room(const Sizes &s, bool own_dz, int dtype) {
    const bool bf16 = is_bf16(dtype);
    return {own_dz ? rounded(s.rows * padded(s.width, bf16) * (bf16 ? 2 : 4)) : 0,
            std::max(product_bytes(kGradX, s.C, s.rows, s.width, bf16), product_bytes(kGradWeight, s.C, s.width, s.rows, bf16))};
}
constexpr double kManyFlops = 5e9;  // of one product: from here on a copy of grad costs less than what it saves
bool copies_grad(const Sizes &s, int dtype) {
    return s.N % (is_bf16(dtype) ? 8 : 4) != 0 && 2. * s.rows * s.N * s.C >= kManyFlops;
}

int64_t forward_workspace(Kind kind, const Sizes &s, int dtype) {
    Check c(dtype);
    if (!sizes_ok(c, s, DDPM_ACT_NONE)) return 0;
    return product_bytes(kind, s.N, s.rows, s.C, is_bf16(dtype));
}

int forward(Kind kind, const void *x, const void *weight, const void *bias, const void *residual, void *y, float *saved,
            void *workspace, const Sizes &s, int64_t x_row, int64_t residual_row, int activation, int dtype,
            hipStream_t stream) {
    Check c(dtype);
    if (!sizes_ok(c, s, activation)) return DDPM_ERR_INVALID_ARG;
    c.stride(x_row);
    if (residual != nullptr) c.stride(residual_row);
    if (c.bad) return DDPM_ERR_INVALID_ARG;
    c.input(x, extent(1, s.rows, s.C, 0, x_row), c.es());
    c.input(weight, (double)s.width * s.C, c.es());
    c.maybe_in(bias, s.width, c.es());
    if (residual != nullptr) c.input(residual, extent(1, s.rows, s.N, 0, residual_row), c.es());
    c.output(y, (double)s.rows * s.N, c.es());
    c.maybe_out(saved, (double)s.rows * s.width, 4);
    const int64_t room = forward_workspace(kind, s, dtype);
    if (room > 0) c.workspace(workspace, (double)room);
    const int st = c.done();
    if (st != DDPM_OK) return st;
    Product a = {};
    a.p = weight;
    a.q = x;
    a.p_ld = s.C;
    a.q_ld = x_row;
    a.np = s.N;
    a.nq = s.rows;
    a.nk = s.C;
    a.out = y;
    a.saved = saved;
    a.bias = bias;
    a.residual = residual;
    a.residual_ld = residual_row;
    a.act = activation;
    (void)hipGetLastError();
    return status_of(launch_product(kind, a, workspace, is_bf16(dtype), stream));
}

int64_t backward_workspace(const Sizes &s, bool through, int activation, int dtype) {
    Check c(dtype);
    return sizes_ok(c, s, activation) ? backward_room(s, through || copies_grad(s, dtype), dtype).all() : 0;
}

int backward(bool gated, const void *grad, const void *x, const void *weight, const float *saved, void *grad_x,
             void *grad_weight, void *grad_bias, void *workspace, const Sizes &s, int64_t x_row, int64_t grad_row,
             int activation, int dtype, hipStream_t stream) {
    Check c(dtype);
    if (!sizes_ok(c, s, activation) || (grad_weight == nullptr) != (grad_bias == nullptr)) return DDPM_ERR_INVALID_ARG;
    c.stride(x_row);
    c.stride(grad_row);
    if (c.bad) return DDPM_ERR_INVALID_ARG;
    const bool through = gated || activation != DDPM_ACT_NONE, own_dz = through || copies_grad(s, dtype), bf16 = is_bf16(dtype);
    c.input(grad, extent(1, s.rows, s.N, 0, grad_row), c.es());
    c.input(x, extent(1, s.rows, s.C, 0, x_row), c.es());
    c.input(weight, (double)s.width * s.C, c.es());
    if (through) c.input(saved, (double)s.rows * s.width, 4);
    c.maybe_out(grad_x, (double)s.rows * s.C, c.es());
    c.maybe_out(grad_weight, (double)s.width * s.C, c.es());
    c.maybe_out(grad_bias, s.width, c.es());
    const Room room = backward_room(s, own_dz, dtype);
    if (room.all() > 0) c.workspace(workspace, (double)room.all());
    const int st = c.done();
    if (st != DDPM_OK) return st;
    (void)hipGetLastError();
    Product a = {};
    a.q = grad;
    a.q_ld = grad_row;
    if (own_dz) {
        const hipError_t e = through ? launch_dz(gated, grad, grad_row, saved, workspace, s.rows, s.N, activation, bf16, stream)
                                     : launch_copies({grad, grad_row, s.rows, s.N, workspace}, {}, bf16, stream);
        if (e != hipSuccess) return status_of(e);
        a.q = workspace;
        a.q_ld = padded(s.width, bf16);
        a.q_padded = true;
    }
    void *rest = (char *)workspace + room.dz;
    if (grad_x != nullptr) {
        Product b = a;
        b.p = weight;
        b.p_ld = s.C;
        b.np = s.C;
        b.nq = s.rows;
        b.nk = s.width;
        b.out = grad_x;
        const hipError_t e = launch_product(kGradX, b, rest, bf16, stream);
        if (e != hipSuccess) return status_of(e);
    }
    if (grad_weight != nullptr) {
        a.p = x;
        a.p_ld = x_row;
        a.np = s.C;
        a.nq = s.width;
        a.nk = s.rows;
        a.out = grad_weight;
        a.sums = grad_bias;
        const hipError_t e = launch_product(kGradWeight, a, rest, bf16, stream);
        if (e != hipSuccess) return status_of(e);
    }
    return DDPM_OK;
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

int64_t ddpm_linear_bwd_workspace(int64_t rows, int64_t C, int64_t N, int activation, int dtype) {
    return backward_workspace({rows, C, N, N}, activation != DDPM_ACT_NONE, activation, dtype);
}

int ddpm_linear_bwd(const void *grad, const void *x, const void *weight, const float *saved, void *grad_x,
                    void *grad_weight, void *grad_bias, void *workspace, int64_t rows, int64_t C, int64_t N, int64_t x_row,
                    int64_t grad_row, int activation, int dtype, hipStream_t stream) {
    return backward(false, grad, x, weight, saved, grad_x, grad_weight, grad_bias, workspace, {rows, C, N, N}, x_row, grad_row,
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

int64_t ddpm_gated_linear_bwd_workspace(int64_t rows, int64_t C, int64_t N, int dtype) {
    return backward_workspace({rows, C, N, 2 * N}, true, DDPM_ACT_NONE, dtype);
}

int ddpm_gated_linear_bwd(const void *grad, const void *x, const void *weight, const float *saved, void *grad_x,
                          void *grad_weight, void *grad_bias, void *workspace, int64_t rows, int64_t C, int64_t N,
                          int64_t x_row, int64_t grad_row, int activation, int dtype, hipStream_t stream) {
    return backward(true, grad, x, weight, saved, grad_x, grad_weight, grad_bias, workspace, {rows, C, N, 2 * N}, x_row, grad_row,
                    activation, dtype, stream);
}

}  // extern "C"
