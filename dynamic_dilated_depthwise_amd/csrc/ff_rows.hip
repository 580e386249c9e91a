// ff_rows.hip -- the forward products of few rows (a decoding batch's tokens): bound by reading the
// weights once.  A workgroup has 16 rows of the weight (gated: 16 of each half) and all rows of x; its
// waves take runs of the contraction in turn, straight from memory into matrix operands, the next run's
// loads under way while one is multiplied, and their sums are joined in LDS, wave after wave.
#include "ff_gemm.hpp"

namespace ddpm {
namespace ff {

namespace {

constexpr int kMostWaves = 8;

// A run of the contraction: PARTS fragments of 32 for each of the operands' 16 rows.
template <typename T, int SETS, int PARTS>
struct Run {
    static constexpr int kVecs = 32 / 4 / kVec<T>, kLong = 32 * PARTS;  // vectors of a lane in a fragment
    u32x4 r[SETS][PARTS][kVecs];
    __device__ __forceinline__ void load(const T *const (&row)[SETS], int64_t k, int64_t nk, int g) {
        if (k + kLong <= nk) {
#pragma unroll
            for (int s = 0; s < SETS; ++s)
#pragma unroll
                for (int i = 0; i < PARTS; ++i)
#pragma unroll
                    for (int v = 0; v < kVecs; ++v) r[s][i][v] = *(const u32x4_a2 *)(row[s] + k + 32 * i + 8 * g + v * kVec<T>);
        } else {
#pragma unroll
            for (int s = 0; s < SETS; ++s)
#pragma unroll
                for (int i = 0; i < PARTS; ++i)
#pragma unroll
                    for (int v = 0; v < kVecs; ++v) {
                        const int64_t at = k + 32 * i + 8 * g + v * kVec<T>;
                        r[s][i][v] = load_vec<T>(row[s] + (at < nk ? at : 0), nk - at);
                    }
        }
    }
    __device__ __forceinline__ Frag<T> get(int s, int i) const {
        if constexpr (Elem<T>::is_bf16) {
            return __builtin_bit_cast(bf16x8, r[s][i][0]);
        } else {
            FragF f;
#pragma unroll
            for (int e = 0; e < 8; ++e) f.v[e] = __uint_as_float(r[s][i][e / 4][e % 4]);
            return f;
        }
    }
};

// MT: rows of x, in sixteens.
template <typename T, bool GATED, int MT>
__global__ __launch_bounds__(kMostWaves *kWave) void rows_kernel(const Product a) {
    constexpr int kHalves = GATED ? 2 : 1, kParts = (MT > 2 ? 2 : 4) * (Elem<T>::is_bf16 ? 2 : 1) / 2, kLd = 20;
    __shared__ float red[kMostWaves][kHalves * MT][16][kLd];
    const int tid = threadIdx.x, wave = wave_of(tid), waves = blockDim.x / kWave, l16 = tid % 16, g = tid % kWave / 16;
    const int64_t p0 = (int64_t)blockIdx.x * 16;
    const T *w[kHalves], *x[MT];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {  // rows that are not there: the last one, whose sums nobody takes
        const int64_t p = p0 + l16 < a.np ? p0 + l16 : a.np - 1;
        w[h] = (const T *)a.p + (p + h * a.np) * a.p_ld;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int64_t q = 16 * m + l16 < a.nq ? 16 * m + l16 : a.nq - 1;
        x[m] = (const T *)a.q + q * a.q_ld;
    }
    f32x4 acc[kHalves][MT];
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[h][m] = f32x4{0.f, 0.f, 0.f, 0.f};

    typedef Run<T, kHalves, kParts> RunW;
    typedef Run<T, MT, kParts> RunX;
    const int64_t stride = (int64_t)waves * RunW::kLong;
    int64_t k = (int64_t)wave * RunW::kLong;
    RunW wn;
    RunX xn;
    if (k < a.nk) {
        wn.load(w, k, a.nk, g);
        xn.load(x, k, a.nk, g);
    }
    for (; k < a.nk; k += stride) {
        const RunW wc = wn;
        const RunX xc = xn;
        if (k + stride < a.nk) {
            wn.load(w, k + stride, a.nk, g);
            xn.load(x, k + stride, a.nk, g);
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i)
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[h][m] = mma(wc.get(h, i), xc.get(m, i), acc[h][m]);
    }
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int m = 0; m < MT; ++m) *(f32x4 *)&red[wave][h * MT + m][l16][4 * g] = acc[h][m];
    __syncthreads();
    // eight columns of a row each
    for (int i = tid; i < 32 * MT; i += (int)blockDim.x) {
        const int q = i / 2, c = i % 2 * 8;
        float v[8], u[8], b[8], bu[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = u[e] = 0.f;
        for (int s = 0; s < waves; ++s) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] += red[s][q / 16][q % 16][c + e];
                if constexpr (GATED) u[e] += red[s][MT + q / 16][q % 16][c + e];
            }
        }
        bias8<T>(a, p0 + c, 0, b);
        if (q == 0) keep8(a, p0 + c, 0, b);
        if constexpr (GATED) {
            bias8<T>(a, p0 + c, 1, bu);
            if (q == 0) keep8(a, p0 + c, 1, bu);
            finish_gated<T>(a, q, p0 + c, v, u, b, bu);
        } else {
            finish_linear<T>(a, q, p0 + c, v, b);
        }
    }
}

template <typename T, bool GATED>
hipError_t rows_of(const Product &a, hipStream_t stream) {
    const int64_t blocks = (a.np + 15) / 16, runs = (a.nk + 127) / 128;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    int waves = 1;
    while (waves < kMostWaves && waves < runs) waves *= 2;
    const dim3 grid((unsigned)blocks), threads(waves * kWave);
    const int64_t m = (a.nq + 15) / 16;
#define X(MT) \
    if (m <= MT) { hipLaunchKernelGGL((rows_kernel<T, GATED, MT>), grid, threads, 0, stream, a); return hipGetLastError(); }
    X(1) X(2) X(3) X(4)
#undef X
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_rows(bool gated, const Product &a, bool bf16, hipStream_t stream) {
    if (bf16) return gated ? rows_of<bf16_t, true>(a, stream) : rows_of<bf16_t, false>(a, stream);
    return gated ? rows_of<float, true>(a, stream) : rows_of<float, false>(a, stream);
}

}  // namespace ff
}  // namespace ddpm
