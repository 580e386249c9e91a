// ff_plan.hpp -- which kernels a call of the feed-forward operators takes, and the room it needs: arithmetic on
// sizes, on the host, so that it compiles without a GPU's compiler too.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "../../include/ddpm_ff.h"

namespace ddpm {
namespace ff {

// y, the gated projection's y, grad_x, grad_W
enum Kind { kForward, kGatedForward, kGradX, kGradWeight };

// Rows of whole 128-byte lines, their last 16-byte chunk filled up with zeros: copies of an operand
// whose rows would otherwise start anywhere.
constexpr int64_t padded(int64_t cols, bool bf16) { return (cols + (bf16 ? 63 : 31)) / (bf16 ? 64 : 32) * (bf16 ? 64 : 32); }

// The tiles that a call may take: waves in p and q, fragments of a wave in p and q, stages, workgroups
// of a compute unit, and the microseconds of a step of the contraction: of one workgroup's share where
// every unit is full, and where every unit has one.
struct Form {
    int wp, wq, mp, nq, stages, per_cu;
    double busy, alone;
    constexpr int kp() const { return wp * mp * 16; }
    constexpr int kq() const { return wq * nq * 16; }
};
constexpr int kFormCount = 5, kGeneral = 1;  // kGeneral: the one for operands that cannot go straight to LDS
// bfloat16: as many waves as registers allow, so that one's reads of LDS run behind another's products
// (256 x 256 with 16 waves 798 us at 8192^3, with 8 848; 128 x 128 with 8 1103, with 4 1370).  Where both
// operands are read by columns 16 waves do not hold their addresses (1129 us, with 8 872).
// float32: waves with large tiles, which split their operands for more products (256 x 256 with 8 waves
// 609 us at 4096^3; before the split took pairs 692, with 16 1115; 128 x 128 with 4 766, with 8 1041).
// Stages: of LDS that steps' chunks are under way to or in; more than two where the tile leaves room and
// a step is shorter than its loads' way (512 x 2048 x 2048 with 128 x 32: 16 -> 12 us with four).
constexpr Form form_of(bool bf16, Kind kind, int k) {
    constexpr Form low[] = {{4, 4, 4, 4, 2, 1, 0, 0},   // 256 x 256
                            {4, 2, 2, 4, 2, 2, 0, 0},   // 128 x 128
                            {2, 4, 2, 4, 2, 2, 0, 0},   // 64 x 256: results of few columns
                            {4, 1, 2, 4, 3, 2, 0, 0},   // 128 x 64
                            {4, 1, 2, 2, 4, 2, 0, 0}};  // 128 x 32: few rows
    constexpr Form full[] = {{2, 4, 8, 4, 2, 1, 0, 0}, {2, 2, 4, 4, 2, 2, 0, 0}, {1, 4, 4, 4, 2, 2, 0, 0}, {4, 1, 2, 4, 3, 2, 0, 0},
                             {4, 1, 2, 2, 4, 2, 0, 0}};
    // Of 256 tiles and of 512 (256 where one fits), the difference between 72 steps and 24 (float32's before its
    // splits held operands to bfloat16's range, 4 % in every form).
    constexpr double times[2][3][5][2] = {{{{4.56, 4.56}, {1.32, 1.55}, {1.35, 1.59}, {0.81, 0.95}, {0.50, 0.62}},    // float32: y
                                           {{4.45, 4.45}, {1.32, 1.45}, {1.36, 1.68}, {0.81, 0.96}, {0.50, 0.65}},    // grad_x
                                           {{4.60, 4.60}, {1.31, 1.67}, {1.39, 1.70}, {0.86, 1.29}, {0.57, 0.85}}},   // grad_W
                                          {{{1.55, 1.55}, {0.45, 0.68}, {0.52, 0.77}, {0.28, 0.40}, {0.22, 0.26}},    // bfloat16
                                           {{1.53, 1.53}, {0.45, 0.73}, {0.51, 0.77}, {0.27, 0.39}, {0.24, 0.31}},
                                           {{1.55, 1.55}, {0.50, 0.84}, {0.51, 0.85}, {0.29, 0.50}, {0.27, 0.37}}}};
    Form f = bf16 ? low[k] : full[k];
    if (bf16 && kind == kGradWeight && k == 0) f.wp = 2, f.mp = 8;
    const int row = kind == kGradX ? 1 : kind == kGradWeight ? 2 : 0;
    f.busy = times[bf16][row][k][0];
    f.alone = times[bf16][row][k][1];
    return f;
}

// How a call is cut.  The tiles of the last round of workgroups, which would leave compute units idle,
// are cut along the contraction into pieces that fill them, where the way of the pieces' results
// through memory and the second kernel that joins them cost less than what that saves.
struct Cut {
    int form = 0, pieces = 1;
    int64_t tiles_p = 0, tiles_q = 0, whole = 0, run = 0;
    double cost = 0.;  // microseconds
    int64_t slots() const { return (tiles_p * tiles_q - whole) * pieces; }
};
constexpr int64_t kUnits = 256;       // compute units
// Lanes that share the pieces of eight neighbouring columns where they are joined.
constexpr int finish_lanes(int pieces) { return pieces >= 64 ? 32 : pieces >= 16 ? 8 : pieces >= 4 ? 2 : 1; }
constexpr int kLeastSteps = 2;        // of a piece
constexpr double kBytes = 4.5e6;      // bytes of results a microsecond
constexpr double kSecondKernel = 6.;  // microseconds

inline Cut cut_for(const Form &f, bool bf16, int64_t p, int64_t q, int64_t steps) {
    Cut c;
    c.tiles_p = (p + f.kp() - 1) / f.kp();
    c.tiles_q = (q + f.kq() - 1) / f.kq();
    const double tiles = (double)c.tiles_p * (double)c.tiles_q, area = (double)f.kp() * f.kq();
    const int64_t slots = kUnits * f.per_cu;
    // a step of m workgroups on a unit; n workgroups of so many steps: whole rounds, and what the last
    // one has on the fullest unit
    const auto step = [&](int64_t m) { return m == 0 ? 0. : m * f.busy > f.alone ? m * f.busy : f.alone; };
    const auto last = [&](int64_t n) { return (n % slots + kUnits - 1) / kUnits; };
    const auto time = [&](int64_t n, int64_t steps_) { return steps_ * ((double)(n / slots) * step(f.per_cu) + step(last(n))); };
    const double out = area * (bf16 ? 2 : 4) / kBytes, part = area * 8 / kBytes;
    const int64_t n = (int64_t)(tiles < 4e9 ? tiles : 4e9);
    c.whole = n;
    c.cost = time(n, steps) + n * out;
    for (const int64_t round : {slots, kUnits}) {
        const int64_t rest = n % round, whole = n - rest, beside = f.per_cu - last(whole);
        if (n >= 16 * slots) break;
        for (int s = 2; rest && s <= 256 && (steps + s - 1) / s >= kLeastSteps; ++s) {
            const int64_t run = (steps + s - 1) / s, m = (rest * s + kUnits - 1) / kUnits;
            // pieces that find room beside the last round's whole tiles run with them
            const double t = (last(whole) != 0 && m <= beside ? time(whole, steps) + run * (step(last(whole) + m) - step(last(whole)))
                                                              : time(whole, steps) + time(rest * s, run)) +
                             n * out + kSecondKernel + rest * s * part;
            if (t < c.cost) {
                c.cost = t;
                c.pieces = s;
                c.whole = whole;
            }
        }
    }
    return c;
}

inline Cut cut_of(Kind kind, int64_t np, int64_t nq, int64_t nk, int terms, bool bf16, bool direct) {
    const int64_t step = bf16 ? 64 : 32, p = kind == kGatedForward ? 2 * np : np, steps = (nk + step - 1) / step;
    Cut best;
    for (int k = 0; k < kFormCount; ++k) {
        if (!direct && k != kGeneral) continue;
        Form f = form_of(bf16, kind, k);
        f.busy *= terms;  // a step of each term
        f.alone *= terms;
        Cut c = cut_for(f, bf16, p, nq, steps);
        c.form = k;
        if (best.tiles_p == 0 || c.cost < best.cost) best = c;
    }
    best.run = (steps + best.pieces - 1) / best.pieces * step;
    best.pieces = (int)((nk + best.run - 1) / best.run);  // none is empty
    return best;
}

constexpr int64_t kMostRows = 64;  // of the kernels for few rows
// Whether the forward takes a kernel of few rows (ff_rows.hip): for operands that cannot go straight to LDS
// the one of any alignment, else the chunked one.  That reads all of x for each 16 columns of the result, so
// it is for few of them, or for little of x.  Microseconds, chunked and tiles (calls behind one another).  bfloat16: 48 rows of 5632 to
// 2048 9.1, 15.1, of 512 to 8192 6.3, 5.4; 24 of 2048 to 5632 6.9, 11.1, to 32000 29.8, 20.7; one of 2048 to
// 5632 5.3, 9, to 16384 15.0, 12.2.  float32, which is split at each read (4 to 7 % more since the splits hold
// operands to bfloat16's range): 24 of 2048 to 5632 16.2, 19.3,
// of 16384 to 512 44.5, 28.1; 48 of 4096 to 4096 21.5, 27.1, of 5632 to 2048 23.4, 22.0; 64 of 1024 to 2304
// 9.3, 12.2, of 2048 to 5632 29.5, 23.6.
inline bool few_rows(Kind kind, int64_t np, int64_t nq, int64_t nk, bool bf16, bool direct) {
    if ((kind != kForward && kind != kGatedForward) || nq > kMostRows) return false;
    if (!direct) return true;
    const int64_t blocks = (np + 15) / 16;
    if (bf16) return blocks <= (nq <= 32 ? 512 : 256);
    return nq <= 16 || (blocks <= 512 && nk <= (nq <= 32 ? 8192 : nq <= 48 ? 4096 : 1024));
}

// Bytes of the pieces' results.
inline int64_t part_bytes(bool bf16, Kind kind, const Cut &c) {
    if (c.pieces == 1) return 0;
    const Form f = form_of(bf16, kind, c.form);
    const int64_t kp = f.kp(), kq = f.kq();
    return c.slots() * (kp * kq + (kind == kGradWeight ? kq : 0)) * 4;
}

// Bytes that launch_product needs at `work` (for these sizes, any strides and alignment); terms: of Q, one or two.
inline int64_t product_bytes(Kind kind, int64_t np, int64_t nq, int64_t nk, int terms, bool bf16) {
    int64_t most = 0;
    for (const bool direct : {false, true}) {
        if (few_rows(kind, np, nq, nk, bf16, direct)) continue;
        most = std::max(most, part_bytes(bf16, kind, cut_of(kind, np, nq, nk, terms, bf16, direct)));
    }
    return most;
}

// Microseconds of a product, straight to LDS or not, as far as its cut foresees.
inline double product_time(Kind kind, int64_t np, int64_t nq, int64_t nk, int terms, bool bf16, bool straight) {
    const double t = cut_of(kind, np, nq, nk, terms, bf16, straight).cost;
    // The form for any alignment takes 1.7 times as long with both operands along their rows, and 3.3 and
    // 5.5 times with one and both read by columns (bfloat16, products of 4095^3; float32 1.1 to 1.4).
    return straight ? t : t * (!bf16 ? 1.25 : kind == kGradX ? 3.3 : kind == kGradWeight ? 5.5 : 1.7);
}

// Those of copies of so many bytes.
inline double copies_time(int64_t bytes) { return 5. + 2. * (double)bytes / kBytes; }

// The backward of few channels in one kernel (ff_small.hip): rows of a tile, workgroups (as many as fit the chip, each
// with rows to work on), bytes of their partials.
constexpr int kSmallCols = 64, kSmallWidth = 256;
constexpr int small_rows(bool bf16) { return bf16 ? 64 : 32; }
inline bool small_backward(int64_t C, int64_t width) { return C <= kSmallCols && width <= kSmallWidth; }
inline int small_groups(int64_t rows, bool bf16) {
    const int64_t tiles = (rows + small_rows(bf16) - 1) / small_rows(bf16);
    return (int)(tiles < kUnits ? tiles : kUnits);
}
inline int64_t small_bytes(int64_t rows, int64_t C, int64_t width, bool bf16) { return small_groups(rows, bf16) * (width * C + width) * 4; }

// Sizes of a call: x [rows, C], y [rows, N], `width` = N or 2 N columns of z.
struct Sizes {
    int64_t rows, C, N, width;
};

inline int64_t rounded(int64_t bytes) { return (bytes + 255) / 256 * 256; }
inline int64_t element(bool bf16) { return bf16 ? 2 : 4; }
inline int64_t chunk(bool bf16) { return 16 / element(bf16); }

// What the forward saves for an activation's or a gate's backward: z in float32, or, with few columns of
// x and more of z than the caches hold, its bias alone, and the backward makes z again (training 16384
// rows to 2 2048 columns, bfloat16, microseconds with z saved and made again: C = 256 434, 396; 768
// 685, 691; 1536 1064, 1144; one half with gelu: 512 315, 306; 768 369, 376; 65536 rows to 2 128 in
// float32: 72 139, 133; 128 149, 150.  Where z stays in the caches both are the same up to C = 256 and
// saving is faster beyond).
// Backwards of few channels (ff_small.hip) always make it again, on the chip.
inline bool makes_again(const Sizes &s, bool bf16) {
    if (small_backward(s.C, s.width)) return true;
    const int64_t most = !bf16 ? 96 : s.width == s.N ? 512 : 768;
    return s.C <= most && (double)s.rows * s.width >= 12e6;
}
inline int64_t saved_floats(const Sizes &s, bool through, bool bf16) { return !through ? 0 : makes_again(s, bf16) ? s.width : s.rows * s.width; }

// x and weight, whose rows of C elements are no whole chunks, as copies with rows that are, where those
// cost less than the products' form for any alignment.
inline int64_t x_copy_bytes(const Sizes &s, bool bf16) { return rounded(s.rows * padded(s.C, bf16) * element(bf16)); }
inline int64_t weight_copy_bytes(const Sizes &s, bool bf16) { return rounded(s.width * padded(s.C, bf16) * element(bf16)); }
inline double forward_time(Kind kind, const Sizes &s, bool bf16, bool straight) {
    return product_time(kind, s.N, s.rows, s.C, 1, bf16, straight);
}
// The same of few rows: nanoseconds of an element of the contraction, as measured with 1 to 64 rows and C from
// 256 to 5632 (with copies at hand at least the weight's way).  Rows of odd length, straight and by copies,
// microseconds: bfloat16 64 rows of 5633 to 128 85, 13, 24 of 4097 to 4096 35, 25, one 17, 23; float32 64 of
// 5633 to 128 51, 26, of 4097 to 4096 39, 60.
inline double rows_time(Kind kind, const Sizes &s, bool bf16, bool straight) {
    const double halves = kind == kGatedForward ? 2. : 1., k = s.C * 1e-3, weight = (double)weight_copy_bytes(s, bf16) / 5e6;
    if (straight) return 4. + std::max(k * (bf16 ? 0.2 * halves + 0.013 * s.rows : 1.5 * halves + 0.04 * s.rows), weight);
    return 4. + k * (bf16 ? 3. * halves + 0.18 * s.rows : 2. * halves + 0.1 * s.rows) * std::max(1., s.N / 8192.);
}
inline bool forward_copies(Kind kind, const Sizes &s, bool bf16) {
    if (s.C % chunk(bf16) == 0) return false;
    const double copies = copies_time(x_copy_bytes(s, bf16) + weight_copy_bytes(s, bf16));
    if (s.rows <= kMostRows) return copies + rows_time(kind, s, bf16, true) < rows_time(kind, s, bf16, false);
    return forward_time(kind, s, bf16, true) + copies < forward_time(kind, s, bf16, false);
}
inline bool backward_copies(Kind kind, const Sizes &s, bool again, int terms, bool bf16) {
    if (s.C % chunk(bf16) == 0) return false;
    const auto all = [&](bool straight) {
        return product_time(kGradX, s.C, s.rows, s.width, terms, bf16, straight) +
               product_time(kGradWeight, s.C, s.width, s.rows, terms, bf16, straight) + (again ? forward_time(kind, s, bf16, straight) : 0.);
    };
    return all(true) + copies_time(x_copy_bytes(s, bf16) + weight_copy_bytes(s, bf16)) < all(false);
}

// What the backward has in its workspace: dz, where it is another tensor than grad (behind an activation
// or a gate, and where grad's rows are no whole chunks and many enough), copies, the products' pieces.
struct Room {
    bool small, own_dz, copies, again;
    int64_t dz, low, all;  // dz's bytes, elements to its second term (or 0), all bytes
};
// Whether dz has more bits than the type: behind relu alone it is grad or zero.
inline bool two_terms(Kind kind, bool through, int activation, bool bf16) {
    return through && bf16 && (kind == kGatedForward || activation != DDPM_ACT_RELU);
}
constexpr double kManyFlops = 5e9;  // of one product: from here on a copy of grad costs less than what it saves
inline Room backward_room(Kind kind, const Sizes &s, bool through, int activation, bool bf16) {
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

}  // namespace ff
}  // namespace ddpm
