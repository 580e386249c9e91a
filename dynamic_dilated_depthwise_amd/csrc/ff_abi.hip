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
int64_t element(bool bf16) { return bf16 ? 2 : 4; }
int64_t chunk(bool bf16) { return 16 / element(bf16); }

// What the forward saves for an activation's or a gate's backward: z in float32, or, with few columns of
// x and more of z than the caches hold, its bias alone, and the backward makes z again (training 16384
// rows to 2 2048 columns, bfloat16, microseconds with z saved and made again: C = 256 323, 227; 768
// 472, 419; 1536 750, 780; one half with gelu: 512 220, 213; 768 266, 275; 65536 rows to 2 128 in
// float32: 64 114, 105; 128 143, 143.  Where z stays in the caches both are the same up to C = 256 and
// saving is faster beyond).
// Backwards of few channels (ff_small.hip) always make it again, on the chip.
bool makes_again(const Sizes &s, bool bf16) {
    if (small_backward(s.C, s.width)) return true;
    const int64_t most = !bf16 ? 96 : s.width == s.N ? 512 : 768;
    return s.C <= most && (double)s.rows * s.width >= 12e6;
}
int64_t saved_floats(const Sizes &s, bool through, bool bf16) { return !through ? 0 : makes_again(s, bf16) ? s.width : s.rows * s.width; }

// x and weight, whose rows of C elements are no whole chunks, as copies with rows that are, where those
// cost less than the products' form for any alignment.
int64_t x_copy_bytes(const Sizes &s, bool bf16) { return rounded(s.rows * padded(s.C, bf16) * element(bf16)); }
int64_t weight_copy_bytes(const Sizes &s, bool bf16) { return rounded(s.width * padded(s.C, bf16) * element(bf16)); }
double forward_time(Kind kind, const Sizes &s, bool bf16, bool straight) {
    return product_time(kind, s.N, s.rows, s.C, 1, bf16, straight);
}
// The same of few rows: nanoseconds of an element of the contraction, as measured with 1 to 64 rows and C from
// 256 to 5632 (with copies at hand at least the weight's way).  Rows of odd length, straight and by copies,
// microseconds: bfloat16 64 rows of 5633 to 128 85, 13, 24 of 4097 to 4096 35, 25, one 17, 23; float32 64 of
// 5633 to 128 51, 26, of 4097 to 4096 39, 60.
double rows_time(Kind kind, const Sizes &s, bool bf16, bool straight) {
    const double halves = kind == kGatedForward ? 2. : 1., k = s.C * 1e-3, weight = (double)weight_copy_bytes(s, bf16) / 5e6;
    if (straight) return 4. + std::max(k * (bf16 ? 0.2 * halves + 0.013 * s.rows : 1.5 * halves + 0.04 * s.rows), weight);
    return 4. + k * (bf16 ? 3. * halves + 0.18 * s.rows : 2. * halves + 0.1 * s.rows) * std::max(1., s.N / 8192.);
}
bool forward_copies(Kind kind, const Sizes &s, bool bf16) {
    if (s.C % chunk(bf16) == 0) return false;
    const double copies = copies_time(x_copy_bytes(s, bf16) + weight_copy_bytes(s, bf16));
    if (s.rows <= kMostRows) return copies + rows_time(kind, s, bf16, true) < rows_time(kind, s, bf16, false);
    return forward_time(kind, s, bf16, true) + copies < forward_time(kind, s, bf16, false);
}
bool backward_copies(Kind kind, const Sizes &s, bool again, int terms, bool bf16) {
    if (s.C % chunk(bf16) == 0) return false;
    const auto all = [&](bool straight) {
        return product_time(kGradX, s.C, s.rows, s.width, terms, bf16, straight) +
               product_time(kGradWeight, s.C, s.width, s.rows, terms, bf16, straight) + (again ? forward_time(kind, s, bf16, straight) : 0.);
    };
    return all(true) + copies_time(x_copy_bytes(s, bf16) + weight_copy_bytes(s, bf16)) < all(false);
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

// What the backward has in its workspace: dz, where it is another tensor than grad (behind an activation
// or a gate, and where grad's rows are no whole chunks and many enough), copies, the products' pieces.
struct Room {
    bool small, own_dz, copies, again;
    int64_t dz, low, all;  // dz's bytes, elements to its second term (or 0), all bytes
};
// Whether dz has more bits than the type: behind relu alone it is grad or zero.
bool two_terms(Kind kind, bool through, int activation, bool bf16) {
    return through && bf16 && (kind == kGatedForward || activation != DDPM_ACT_RELU);
}
constexpr double kManyFlops = 5e9;  // of one product: from here on a copy of grad costs less than what it saves
Room backward_room(Kind kind, const Sizes &s, bool through, int activation, bool bf16) {
    Room r = {};
    r.small = through && small_backward(s.C, s.width);
    if (r.small) {
        r.all = small_bytes(s.rows, s.C, s.width, bf16);
        return r;
    }
    r.own_dz = through || (s.N % chunk(bf16) != 0 && 2. * s.rows * s.N * s.C >= kManyFlops);
    r.again = through && makes_again(s, bf16);
    const int terms = two_terms(kind, through, activation, bf16) ? 2 : 1;
    const int64_t dz = s.rows * padded(s.width, bf16);
    r.copies = backward_copies(kind, s, r.again, terms, bf16);
    r.dz = r.own_dz ? rounded(terms * dz * element(bf16)) : 0;
    r.low = terms == 2 ? dz : 0;
    int64_t part = std::max(product_bytes(kGradX, s.C, s.rows, s.width, terms, bf16),
                            product_bytes(kGradWeight, s.C, s.width, s.rows, terms, bf16));
    if (r.again) part = std::max(part, product_bytes(kind, s.N, s.rows, s.C, 1, bf16));
    r.all = r.dz + (r.copies ? x_copy_bytes(s, bf16) + weight_copy_bytes(s, bf16) : 0) + part;
    return r;
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
