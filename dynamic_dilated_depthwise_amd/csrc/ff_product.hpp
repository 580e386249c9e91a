// ff_product.hpp -- which form of the tiled product a call takes, for one type; instantiated in a
// source of its own for each type and kind, so that they compile beside each other.
#pragma once

#include "ff_gemm.hpp"

namespace ddpm {
namespace ff {

template <Kind K> struct KindOf;
template <> struct KindOf<kForward> { static constexpr Side sp = kAlong, sq = kAlong; static constexpr Epi e = kLinear; };
template <> struct KindOf<kGatedForward> { static constexpr Side sp = kAlong, sq = kAlong; static constexpr Epi e = kGated; };
template <> struct KindOf<kGradX> { static constexpr Side sp = kDown, sq = kAlong; static constexpr Epi e = kStore; };
template <> struct KindOf<kGradWeight> { static constexpr Side sp = kDown, sq = kDown; static constexpr Epi e = kWeight; };

// Whether an operand can go straight to LDS: whole 16-byte chunks, and a step's tile within a
// buffer's offsets.  rows: those of the tile in memory.
template <typename T>
inline bool direct_ok(Side s, const void *p, int64_t ld, int64_t extent, int64_t nk, int64_t rows, bool padded) {
    constexpr int64_t per = 16 / (int64_t)sizeof(T);
    if ((uintptr_t)p % 16 != 0 || ld % per != 0 || (!padded && (s == kAlong ? nk : extent) % per != 0)) return false;
    return (rows * ld + kStep<T>) * (int64_t)sizeof(T) < (int64_t)kRecords;
}

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
    // Of 256 tiles and of 512 (256 where one fits), the difference between 72 steps and 24.
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

template <typename T>
inline Cut cut_of(Kind kind, int64_t np, int64_t nq, int64_t nk, int terms, bool direct) {
    constexpr bool bf16 = Elem<T>::is_bf16;
    const int64_t p = kind == kGatedForward ? 2 * np : np, steps = (nk + kStep<T> - 1) / kStep<T>;
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
    best.run = (steps + best.pieces - 1) / best.pieces * kStep<T>;
    best.pieces = (int)((nk + best.run - 1) / best.run);  // none is empty
    return best;
}

// Whether the forward takes a kernel of few rows (ff_rows.hip): for operands that cannot go straight to LDS
// the one of any alignment, else the chunked one.  That reads all of x for each 16 columns of the result, so
// it is for few of them, or for little of x.  Microseconds, chunked and tiles.  bfloat16: 48 rows of 5632 to
// 2048 9.1, 15.1, of 512 to 8192 6.3, 5.4; 24 of 2048 to 5632 6.9, 11.1, to 32000 29.8, 20.7; one of 2048 to
// 5632 5.3, 9, to 16384 15.0, 12.2.  float32, which is split at each read: 24 of 2048 to 5632 16.2, 19.3,
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

template <typename G>
hipError_t launch_gemm(Product &a, const Cut &c, hipStream_t stream) {
    const double blocks = (double)c.whole + (double)c.slots();
    if (blocks > 2147483647. || (double)c.tiles_p * (double)c.tiles_q > 2147483647.) return hipErrorInvalidConfiguration;
    a.tiles_p = (uint32_t)c.tiles_p;
    a.tiles_q = (uint32_t)c.tiles_q;
    a.whole = (uint32_t)c.whole;
    a.pieces = c.pieces;
    a.run = c.run;
    hipLaunchKernelGGL((gemm_kernel<G>), dim3((unsigned)blocks), dim3(G::kThreads), 0, stream, a);
    const hipError_t r = hipGetLastError();
    if (r != hipSuccess || c.pieces == 1) return r;
    const int64_t cut = c.tiles_p * c.tiles_q - c.whole;
    hipLaunchKernelGGL((finish_kernel<G>), dim3((unsigned)(cut * (G::kPerTile / (G::kFinishThreads / G::lanes(c.pieces))))), dim3(G::kFinishThreads), 0, stream, a);
    return hipGetLastError();
}

template <typename T, Kind K>
hipError_t product(Product a, void *work, hipStream_t stream) {
    constexpr Side sp = KindOf<K>::sp, sq = KindOf<K>::sq;
    constexpr Epi e = KindOf<K>::e;
    const bool direct = direct_ok<T>(sp, a.p, a.p_ld, a.np, a.nk, K == kGatedForward ? a.np + 256 : 256, a.p_padded) &&
                        direct_ok<T>(sq, a.q, a.q_ld, a.nq, a.nk, 256, a.q_padded);
    if (few_rows(K, a.np, a.nq, a.nk, Elem<T>::is_bf16, direct)) return launch_rows(K == kGatedForward, direct, a, Elem<T>::is_bf16, stream);
    const Cut c = cut_of<T>(K, a.np, a.nq, a.nk, (K == kGradX || K == kGradWeight) && a.low != 0 ? 2 : 1, direct);
    a.part = (float *)work;
#define DDPM_FF_FORM(k, DIRECT)                                                                       \
    if (c.form == k) {                                                                                \
        constexpr Form f = form_of(Elem<T>::is_bf16, K, k);                                           \
        return launch_gemm<Gemm<T, sp, sq, e, f.wp, f.wq, f.mp, f.nq, f.stages, DIRECT>>(a, c, stream);         \
    }
    if (!direct) {
        DDPM_FF_FORM(kGeneral, false)
    } else {
        DDPM_FF_FORM(0, true)
        DDPM_FF_FORM(1, true)
        DDPM_FF_FORM(2, true)
        DDPM_FF_FORM(3, true)
        DDPM_FF_FORM(4, true)
    }
#undef DDPM_FF_FORM
    return hipErrorInvalidValue;
}

}  // namespace ff
}  // namespace ddpm
