// ff_rows.hip -- the forward products of few rows (a decoding batch's tokens): bound by reading the
// weights once.  A workgroup has 16 rows of the weight (gated: 16 of each half) and all rows of x; its
// waves take steps of the contraction in turn and their sums are joined in LDS, wave after wave.  No pieces
// of results go through memory and no second kernel joins them, as the tiles' would.
//
//   chunked_rows_kernel  operands through LDS, whole chunks (one row of 2048 to 2 5632, bfloat16: 8.7 us, 46 MB,
//                        5.3 TB/s; 48 of 5632 to 2048 10.5 us: its 128 workgroups leave half of the units idle)
//   rows_kernel          straight from memory into matrix operands, any alignment (12.6 us; 22 us; weights that
//                        start at odd addresses 33 and 36)
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

constexpr int kRedLd = 20;
template <bool GATED, int MT> using Red = float[(GATED ? 2 : 1) * MT][16][kRedLd];  // a wave's sums in LDS

// The sums of the waves and what follows them.
template <typename T, bool GATED, int MT>
__device__ __forceinline__ void join(const Product &a, Red<GATED, MT> *red, const f32x4 (&acc)[GATED ? 2 : 1][MT], int64_t p0, int wave, int waves) {
    constexpr int kHalves = GATED ? 2 : 1;
    const int tid = threadIdx.x, l16 = tid % 16, g = tid % kWave / 16;
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

// MT: rows of x, in sixteens.
template <typename T, bool GATED, int MT>
__global__ __launch_bounds__(kMostWaves *kWave) void rows_kernel(const Product a) {
    constexpr int kHalves = GATED ? 2 : 1, kParts = (MT > 2 ? 2 : 4) * (Elem<T>::is_bf16 ? 2 : 1) / 2;
    __shared__ __attribute__((aligned(16))) Red<GATED, MT> red[kMostWaves];
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
    join<T, GATED, MT>(a, red, acc, p0, wave, waves);
}


// A step's rows are read in whole lines, eight rows a load, straight to LDS.  A wave has a part of LDS of its
// own, to which the chunks of its next steps are under way while one is multiplied, and waits for nobody
// until the sums are joined.  Two workgroups a compute unit where the waves' steps leave room (bfloat16, one
// row of 2048 to 5632 5.2 us, with one workgroup 7.1); float32, which splits at each read, has eight waves
// first (one row of 5632 to 2 2048 18.4 us, as four and four 22.5).
template <typename T, bool GATED, int MT> constexpr int kRoomOf = (MT <= (Elem<T>::is_bf16 ? 2 : GATED ? 0 : 1) ? 80 : 128) * 1024;
template <typename T, bool GATED, int MT>
struct Chunked {
    static constexpr int kHalves = GATED ? 2 : 1, kStepAll = (kHalves + MT) * 16 * kStepBytes;
    static constexpr int kRoom = kRoomOf<T, GATED, MT>, kWaves = 2 * kStepAll * kMostWaves <= kRoom ? kMostWaves : kMostWaves / 2;
    static constexpr int kStages = kRoom / (kStepAll * kWaves) < 4 ? kRoom / (kStepAll * kWaves) : 4, kLds = kStages * kStepAll * kWaves;
    static constexpr int kLoads = 2 * (kHalves + MT);
    static_assert(kStages >= 2 && sizeof(Red<GATED, MT>) * kWaves <= kLds, "LDS");
};
template <typename T, bool GATED, int MT>
__global__ __launch_bounds__((Chunked<T, GATED, MT>::kWaves) * kWave) void chunked_rows_kernel(const Product a) {
    typedef Chunked<T, GATED, MT> S;
    constexpr int kHalves = S::kHalves, kStages = S::kStages, kPer = kVec<T>;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int tid = threadIdx.x, wave = wave_of(tid), lane = tid % kWave;
    const int64_t p0 = (int64_t)blockIdx.x * 16;
    char *mine = lds + wave * (kStages * S::kStepAll);
    // a load is 8 rows of a step
    const int row = lane / 8, chunk = lane % 8 ^ row;
    uint32_t off_w[2], off_x[2 * MT];
#pragma unroll
    for (int i = 0; i < 2; ++i) off_w[i] = p0 + 8 * i + row < a.np ? (uint32_t)((8 * i + row) * a.p_ld * sizeof(T)) + chunk * 16 : kOutside;
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) off_x[i] = 8 * i + row < a.nq ? (uint32_t)((8 * i + row) * a.q_ld * sizeof(T)) + chunk * 16 : kOutside;
    const T *w = (const T *)a.p + p0 * a.p_ld, *x = (const T *)a.q;
    const int64_t half = a.np * a.p_ld, steps = (a.nk + kStep<T> - 1) / kStep<T>;
    const auto ask = [&](int64_t s, int stage) {
        const int64_t k = s * kStep<T>;
        const bool on = k + chunk * kPer < a.nk;
        char *to = mine + stage * S::kStepAll;
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) load_to_lds(w + h * half + k, on ? off_w[i] : kOutside, to + (2 * h + i) * 1024);
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) load_to_lds(x + k, on ? off_x[i] : kOutside, to + (2 * kHalves + i) * 1024);
    };
    Reader<T, kAlong, 16 * (kHalves + MT)> read;
    read.start(lane);
    f32x4 acc[kHalves][MT];
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[h][m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < kStages - 1; ++t) ask(wave + t * S::kWaves, t);
    int now = 0;
    for (int64_t s = wave; s < steps; s += S::kWaves) {
        const int next = now == 0 ? kStages - 1 : now - 1;
        ask(s + (kStages - 1) * S::kWaves, next);  // past the last step: nothing
        asm volatile("s_waitcnt vmcnt(%0)" :: "n"((kStages - 1) * S::kLoads) : "memory");
        const char *at = mine + now * S::kStepAll;
#pragma unroll
        for (int r = 0; r < kStep<T> / 32; ++r) {
            Operand<T> q[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) q[m] = read.get(at, kHalves + m, r);
#pragma unroll
            for (int h = 0; h < kHalves; ++h) multiply<MT>(acc[h], read.get(at, h, r), q);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read, before it is asked for again
        now = now + 1 == kStages ? 0 : now + 1;
    }
    arrive_but<0>();
    join<T, GATED, MT>(a, (Red<GATED, MT> *)lds, acc, p0, wave, S::kWaves);
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

template <typename T, bool GATED, int MT>
hipError_t chunked(const Product &a, hipStream_t stream) {
    typedef Chunked<T, GATED, MT> S;
    const auto kernel = chunked_rows_kernel<T, GATED, MT>;
    const int64_t blocks = (a.np + 15) / 16;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(S::kWaves * kWave), S::kLds, stream, a);
    return hipGetLastError();
}
template <typename T, bool GATED>
hipError_t chunked_of(const Product &a, hipStream_t stream) {
    const int64_t m = (a.nq + 15) / 16;
#define X(MT) \
    if (m <= MT) return chunked<T, GATED, MT>(a, stream);
    X(1) X(2) X(3) X(4)
#undef X
    return hipErrorInvalidValue;
}

template <typename T>
hipError_t either(bool gated, bool chunked, const Product &a, hipStream_t stream) {
    if (chunked) return gated ? chunked_of<T, true>(a, stream) : chunked_of<T, false>(a, stream);
    return gated ? rows_of<T, true>(a, stream) : rows_of<T, false>(a, stream);
}

}  // namespace

hipError_t launch_rows(bool gated, bool chunked, const Product &a, bool bf16, hipStream_t stream) {
    return bf16 ? either<bf16_t>(gated, chunked, a, stream) : either<float>(gated, chunked, a, stream);
}

}  // namespace ff
}  // namespace ddpm
