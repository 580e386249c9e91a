// ff_point.hip -- the gradient of an activation's or a gate's input, element by element.  Bound by
// memory; a thread takes eight neighbouring columns.
#include "ff_gemm.hpp"

namespace ddpm {
namespace ff {

namespace {

constexpr int kThreads = 256;

// (row, first column) of item i where a row has `per` items.
struct Place {
    int64_t row, col;
};
__device__ __forceinline__ Place place_of(int64_t i, int64_t per) {
    if (i >> 32 == 0) {
        const uint32_t r = (uint32_t)i / (uint32_t)per;
        return {r, ((uint32_t)i - r * (uint32_t)per) * (int64_t)8};
    }
    const int64_t r = i / per;
    return {r, (i - r * per) * 8};
}

template <int ACT> __device__ __forceinline__ void slopes(const float (&z)[8], float (&d)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (ACT == DDPM_ACT_RELU) {
            d[e] = z[e] > 0.f ? 1.f : z[e] <= 0.f ? 0.f : z[e];
        } else if constexpr (ACT == DDPM_ACT_SILU) {
            const float s = 1.f / (1.f + expf(-z[e]));
            d[e] = s * (1.f + z[e] * (1.f - s));
        } else {
            d[e] = 0.5f * erfcf(-0.70710678118654752f * z[e]) + z[e] * 0.39894228040143268f * expf(-0.5f * z[e] * z[e]);
        }
    }
}
__device__ __forceinline__ void slope(const float (&z)[8], float (&d)[8], int act) {
    if (act == DDPM_ACT_RELU) {
        slopes<DDPM_ACT_RELU>(z, d);
    } else if (act == DDPM_ACT_SILU) {
        slopes<DDPM_ACT_SILU>(z, d);
    } else if (act == DDPM_ACT_GELU) {
        slopes<DDPM_ACT_GELU>(z, d);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = 1.f;
    }
}

template <typename T, bool GATED>
__global__ __launch_bounds__(kThreads) void dz_kernel(const T *__restrict__ grad, int64_t grad_ld, const float *__restrict__ saved,
                                                      T *__restrict__ dz, int64_t rows, int64_t N, int act) {
    const int64_t per = (N + 7) / 8, all = rows * per, stride = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += stride) {
        const Place at = place_of(i, per);
        const int64_t n = N - at.col;
        float g[8], z[8], d[8];
        read8<T>(grad + at.row * grad_ld + at.col, n, g);
        const int64_t o = at.row * (GATED ? 2 * N : N) + at.col;
        read8<float>(saved + o, n, z);
        slope(z, d, act);
        if constexpr (GATED) {
            float u[8];
            read8<float>(saved + o + N, n, u);
            activate(z, act);
#pragma unroll
            for (int e = 0; e < 8; ++e) { d[e] = g[e] * u[e] * d[e]; z[e] = g[e] * z[e]; }
            write8<T>(dz + o, n, d);
            write8<T>(dz + o + N, n, z);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] *= g[e];
            write8<T>(dz + o, n, d);
        }
    }
}

unsigned blocks_for(int64_t rows, int64_t N) {
    const int64_t items = rows * ((N + 7) / 8), blocks = (items + kThreads - 1) / kThreads;
    return (unsigned)(blocks < 8192 ? blocks : 8192);
}

template <typename T>
hipError_t dz_of(bool gated, const void *grad, int64_t grad_ld, const float *saved, void *dz, int64_t rows, int64_t N, int act,
                 hipStream_t stream) {
    const dim3 grid(blocks_for(rows, N)), threads(kThreads);
    if (gated) hipLaunchKernelGGL((dz_kernel<T, true>), grid, threads, 0, stream, (const T *)grad, grad_ld, saved, (T *)dz, rows, N, act);
    else hipLaunchKernelGGL((dz_kernel<T, false>), grid, threads, 0, stream, (const T *)grad, grad_ld, saved, (T *)dz, rows, N, act);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dz(bool gated, const void *grad, int64_t grad_ld, const float *saved, void *dz, int64_t rows, int64_t N,
                     int act, bool bf16, hipStream_t stream) {
    return bf16 ? dz_of<bf16_t>(gated, grad, grad_ld, saved, dz, rows, N, act, stream)
                : dz_of<float>(gated, grad, grad_ld, saved, dz, rows, N, act, stream);
}

}  // namespace ff
}  // namespace ddpm
