// ff_product.hpp -- which form of the tiled product a call takes, for one type; instantiated in a
// source of its own for each type and kind, so that they compile beside each other.
#pragma once

#include "ff_gemm.hpp"
#include "ff_plan.hpp"

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
    hipLaunchKernelGGL((finish_kernel<G>), dim3((unsigned)(cut * (G::kPerTile / (G::kFinishThreads / finish_lanes(c.pieces))))), dim3(G::kFinishThreads), 0, stream, a);
    return hipGetLastError();
}

template <typename T, Kind K>
hipError_t product(Product a, void *work, hipStream_t stream) {
    constexpr Side sp = KindOf<K>::sp, sq = KindOf<K>::sq;
    constexpr Epi e = KindOf<K>::e;
    const bool direct = direct_ok<T>(sp, a.p, a.p_ld, a.np, a.nk, K == kGatedForward ? a.np + 256 : 256, a.p_padded) &&
                        direct_ok<T>(sq, a.q, a.q_ld, a.nq, a.nk, 256, a.q_padded);
    if (few_rows(K, a.np, a.nq, a.nk, Elem<T>::is_bf16, direct)) return launch_rows(K == kGatedForward, direct, a, Elem<T>::is_bf16, stream);
    const Cut c = cut_of(K, a.np, a.nq, a.nk, (K == kGradX || K == kGradWeight) && a.low != 0 ? 2 : 1, Elem<T>::is_bf16, direct);
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
