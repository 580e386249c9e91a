// ff_point.hip -- the gradient of an activation's or a gate's input, element by element, and copies of
// operands to rows of whole chunks.  Bound by memory; a thread takes eight neighbouring columns, or a
// chunk.
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

template <typename T, bool GATED>
__global__ __launch_bounds__(kThreads) void dz_kernel(const T *__restrict__ grad, int64_t grad_ld, const float *__restrict__ saved,
                                                      T *__restrict__ dz, int64_t low, int64_t ld, int64_t rows, int64_t N, int act) {
    const int64_t per = (N + 7) / 8, all = rows * per, stride = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += stride) {
        const Place at = place_of(i, per);
        const int64_t n = N - at.col;
        const T *g = grad + at.row * grad_ld;
        const float *s = saved + at.row * (GATED ? 2 * N : N) + at.col;
        T *o = dz + at.row * ld;
        float z[8], u[8];
        read8<float>(s, n, z);
        if constexpr (GATED) {
            read8<float>(s + N, n, u);
            finish_gated_dz<T>(o, low, at.col, N, g, act, z, u);
        } else {
            finish_dz<T>(o, low, at.col, N, g, act, z);
        }
    }
}

// A wave a row: finding the row of each chunk by a division takes as long as the copy (13 MB in two
// operands 10.8 us, so 9.1).  The last chunk of a row is read ending with the row, without branches.
template <typename T>
__global__ __launch_bounds__(kThreads) void copies_kernel(const Copy a, const Copy b) {
    constexpr int kPer = kVec<T>;
    const int wave = wave_of(threadIdx.x), lane = threadIdx.x % kWave;
    const int64_t stride = (int64_t)gridDim.x * (kThreads / kWave);
    for (int64_t i = (int64_t)blockIdx.x * (kThreads / kWave) + wave; i < a.rows + b.rows; i += stride) {
        const bool first = i < a.rows;
        const int64_t row = first ? i : i - a.rows;
        const int cols = (int)(first ? a.cols : b.cols);
        const T *from = (const T *)(first ? a.src : b.src) + row * (first ? a.ld : b.ld);
        T *to = (T *)(first ? a.dst : b.dst) + row * padded(cols, Elem<T>::is_bf16);
        if (cols > kPer) {
            for (int c = lane * kPer; c < cols; c += kWave * kPer) {
                Raw<T, kPer> r;
                r.template load<kOdd>(from, c, cols, true);
                *(u32x4 *)(to + c) = r.r;
            }
        } else if (lane == 0) {
            *(u32x4 *)to = load_vec<T>(from, cols);
        }
    }
}

unsigned blocks_for(int64_t rows, int64_t N) {
    const int64_t items = rows * ((N + 7) / 8), blocks = (items + kThreads - 1) / kThreads;
    return (unsigned)(blocks < 8192 ? blocks : 8192);
}

template <typename T>
hipError_t dz_of(bool gated, const void *grad, int64_t grad_ld, const float *saved, void *dz, int64_t low, int64_t rows, int64_t N,
                 int act, hipStream_t stream) {
    const dim3 grid(blocks_for(rows, N)), threads(kThreads);
    const int64_t ld = padded(gated ? 2 * N : N, Elem<T>::is_bf16);
    if (gated) hipLaunchKernelGGL((dz_kernel<T, true>), grid, threads, 0, stream, (const T *)grad, grad_ld, saved, (T *)dz, low, ld, rows, N, act);
    else hipLaunchKernelGGL((dz_kernel<T, false>), grid, threads, 0, stream, (const T *)grad, grad_ld, saved, (T *)dz, low, ld, rows, N, act);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dz(bool gated, const void *grad, int64_t grad_ld, const float *saved, void *dz, int64_t low, int64_t rows,
                     int64_t N, int act, bool bf16, hipStream_t stream) {
    return bf16 ? dz_of<bf16_t>(gated, grad, grad_ld, saved, dz, low, rows, N, act, stream)
                : dz_of<float>(gated, grad, grad_ld, saved, dz, low, rows, N, act, stream);
}

hipError_t launch_copies(const Copy &a, const Copy &b, bool bf16, hipStream_t stream) {
    const int64_t blocks = (a.rows + b.rows + kThreads / kWave - 1) / (kThreads / kWave);
    const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192)), threads(kThreads);
    if (bf16) hipLaunchKernelGGL((copies_kernel<bf16_t>), grid, threads, 0, stream, a, b);
    else hipLaunchKernelGGL((copies_kernel<float>), grid, threads, 0, stream, a, b);
    return hipGetLastError();
}

}  // namespace ff
}  // namespace ddpm
