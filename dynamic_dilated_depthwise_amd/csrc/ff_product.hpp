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
inline bool direct_ok(Side s, const void *p, int64_t ld, int64_t extent, int64_t nk, int64_t rows) {
    constexpr int64_t per = 16 / (int64_t)sizeof(T);
    if ((uintptr_t)p % 16 != 0 || ld % per != 0 || (s == kAlong ? nk : extent) % per != 0) return false;
    return (rows * ld + kStep<T>) * (int64_t)sizeof(T) < (int64_t)kRecords;
}

// How a call is cut: the tile and the runs of the contraction.
struct Cut {
    int kp, kq, splits;
    int64_t run;
};
template <typename T>
inline Cut cut_of(Kind kind, int64_t np, int64_t nq, int64_t nk, bool direct) {
    const int64_t p = kind == kGatedForward ? 2 * np : np, steps = (nk + kStep<T> - 1) / kStep<T>;
    const auto tiles = [&](int64_t kp, int64_t kq) { return (double)((p + kp - 1) / kp) * (double)((nq + kq - 1) / kq); };
    Cut c = {128, 128, 1, 0};
    if (direct && Elem<T>::is_bf16 && tiles(256, 256) >= 160) c.kp = c.kq = 256;
    const double t = tiles(c.kp, c.kq);
    // few tiles: the contraction is split until there are two workgroups for each compute unit, but
    // not into runs of less than 8 steps
    if (t < 256 && steps >= 16) {
        int64_t s = (int64_t)(512 / t);
        if (s > steps / 8) s = steps / 8;
        if (s > 1) c.splits = (int)s;
    }
    c.run = (steps + c.splits - 1) / c.splits * kStep<T>;
    c.splits = (int)((nk + c.run - 1) / c.run);
    return c;
}

inline int64_t part_stride(Kind kind, int64_t np, int64_t nq) {
    return (kind == kGatedForward ? 2 * np : np) * nq + (kind == kGradWeight ? nq : 0);
}

template <typename G>
hipError_t launch_gemm(Product &a, const Cut &c, int64_t p, hipStream_t stream) {
    const int64_t tp = (p + G::kP - 1) / G::kP, tq = (a.nq + G::kQ - 1) / G::kQ;
    if ((double)tp * (double)tq * c.splits > 2147483647.) return hipErrorInvalidConfiguration;
    a.tiles_p = (uint32_t)tp;
    a.tiles_q = (uint32_t)tq;
    a.run = c.run;
    hipLaunchKernelGGL((gemm_kernel<G>), dim3((unsigned)(tp * tq * c.splits)), dim3(G::kThreads), 0, stream, a);
    return hipGetLastError();
}

template <typename T, Kind K>
hipError_t product(Product a, float *part, hipStream_t stream) {
    constexpr Side sp = KindOf<K>::sp, sq = KindOf<K>::sq;
    constexpr Epi e = KindOf<K>::e;
    const int64_t p = K == kGatedForward ? 2 * a.np : a.np;
    const bool direct = direct_ok<T>(sp, a.p, a.p_ld, a.np, a.nk, K == kGatedForward ? a.np + 256 : 256) &&
                        direct_ok<T>(sq, a.q, a.q_ld, a.nq, a.nk, 256);
    const Cut c = cut_of<T>(K, a.np, a.nq, a.nk, direct);
    if (c.splits > 1) {
        a.part = part;
        a.part_stride = part_stride(K, a.np, a.nq);
    }
    hipError_t r;
    if (!direct) {
        r = launch_gemm<Gemm<T, sp, sq, e, 2, 2, 4, 4, false>>(a, c, p, stream);
    } else if (c.kp == 256) {
        if constexpr (Elem<T>::is_bf16) r = launch_gemm<Gemm<T, sp, sq, e, 2, 4, 8, 4, true>>(a, c, p, stream);
        else r = hipErrorInvalidConfiguration;
    } else {
        r = launch_gemm<Gemm<T, sp, sq, e, 2, 2, 4, 4, true>>(a, c, p, stream);
    }
    if (r != hipSuccess || c.splits == 1) return r;
    return launch_finish(K, a, c.splits, Elem<T>::is_bf16, stream);
}

}  // namespace ff
}  // namespace ddpm
