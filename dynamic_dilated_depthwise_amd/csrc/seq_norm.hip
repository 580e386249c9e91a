// seq_norm.hip -- layer norm over the last axis, forward and backward, and the sum of
// float32 partials that the weight gradients of the sequence operators share.
//
//   y = (x - mean) * rstd * weight + bias,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   xh = (x - mean) * rstd,  gw = g * weight
//   grad_x = rstd * (gw - mean(gw) - xh * mean(gw * xh))
//   grad_weight = sum over rows of g * xh,   grad_bias = sum over rows of g
//
// Both directions are bound by memory.  A row lives in the registers of a group of lanes
// (16, a wave or a workgroup), so it is read once; the mean is taken first and the
// squares of the differences after it, in float32.  The backward's column sums stay in
// registers over the rows that a workgroup walks, are joined in LDS and leave as one
// float32 row per workgroup; a second short kernel adds those in a fixed order (no
// atomics: results repeat bit for bit).
#include "seq_common.hpp"
#include "seq_launch.hpp"

namespace ddpm {
namespace seq {

constexpr int kThreads = 256;

// Sum over the LPR lanes of a row's group.  LPR <= 64 stays inside the wave.
template <int LPR>
__device__ __forceinline__ float group_sum(float v, float *red) {
#pragma unroll
    for (int m = 1; m < (LPR < kWave ? LPR : kWave); m *= 2) v += __shfl_xor(v, m, kWave);
    if constexpr (LPR > kWave) {
        static_assert(LPR == kThreads, "a group is part of a wave, a wave or the workgroup");
        const int w = threadIdx.x / kWave;
        __syncthreads();
        if (threadIdx.x % kWave == 0) red[w] = v;
        __syncthreads();
        v = red[0] + red[1] + red[2] + red[3];
    }
    return v;
}

// 16381 x 2048 bfloat16: 24 us, 5.6 TB/s; 65536 x 64 float32: 8.6 us, 3.9 TB/s; 7 x 1024
// bfloat16: 2.8 us.
template <typename T, int LPR, int NV, Reach R>
__global__ __launch_bounds__(kThreads) void norm_fwd_kernel(const T *__restrict__ x, const T *__restrict__ weight,
                                                            const T *__restrict__ bias, T *__restrict__ y,
                                                            float *__restrict__ mean, float *__restrict__ rstd,
                                                            int64_t rows, int C, int64_t x_stride, float eps) {
    constexpr int V = kVec<T>, ROWS = kThreads / LPR;
    __shared__ float red[4];
    const int lane = threadIdx.x % LPR;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / LPR;
    const bool on = row < rows;
    const T *xr = x + (on ? row : 0) * x_stride;
    Raw<T, V> v[NV];
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        v[k].template load<R>(xr, (k * LPR + lane) * V, C, on);
#pragma unroll
        for (int e = 0; e < V; ++e) sum += v[k][e];
    }
    const float mu = group_sum<LPR>(sum, red) / (float)C;
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float d = (k * LPR + lane) * V + e < C ? v[k][e] - mu : 0.f;
            sq += d * d;
        }
    const float rs = 1.f / sqrtf(group_sum<LPR>(sq, red) / (float)C + eps);
    if (!on) return;
    if (mean != nullptr && lane == 0) {
        mean[row] = mu;
        rstd[row] = rs;
    }
    T *yr = y + row * C;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * LPR + lane) * V;
        if (c >= C) continue;
        Raw<T, V> w, b;
        float o[V];
        w.template load<R>(weight, c, C, true);
        b.template load<R>(bias, c, C, true);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = (v[k][e] - mu) * rs * w[e] + b[e];
        w.set(o);
        w.template store<R>(yr, c, C);
    }
}

// Rows longer than the registers of a workgroup hold: three passes, the later two mostly
// from the caches (2048 x 20000 float32 forward and backward: 315 us, 2.1 TB/s).
template <typename T, Reach R>
__global__ __launch_bounds__(kThreads) void norm_fwd_long_kernel(const T *__restrict__ x, const T *__restrict__ weight,
                                                                 const T *__restrict__ bias, T *__restrict__ y,
                                                                 float *__restrict__ mean, float *__restrict__ rstd,
                                                                 int64_t rows, int C, int64_t x_stride, float eps) {
    constexpr int V = kVec<T>;
    __shared__ float red[4];
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T *xr = x + row * x_stride;
        Raw<T, V> v, w, b;
        float sum = 0.f, sq = 0.f, o[V];
        for (int c = threadIdx.x * V; c < C; c += kThreads * V) {
            v.template load<R>(xr, c, C, true);
#pragma unroll
            for (int e = 0; e < V; ++e) sum += v[e];
        }
        const float mu = group_sum<kThreads>(sum, red) / (float)C;
        for (int c = threadIdx.x * V; c < C; c += kThreads * V) {
            v.template load<R>(xr, c, C, true);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = c + e < C ? v[e] - mu : 0.f;
                sq += d * d;
            }
        }
        const float rs = 1.f / sqrtf(group_sum<kThreads>(sq, red) / (float)C + eps);
        if (mean != nullptr && threadIdx.x == 0) {
            mean[row] = mu;
            rstd[row] = rs;
        }
        for (int c = threadIdx.x * V; c < C; c += kThreads * V) {
            v.template load<R>(xr, c, C, true);
            w.template load<R>(weight, c, C, true);
            b.template load<R>(bias, c, C, true);
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = (v[e] - mu) * rs * w[e] + b[e];
            v.set(o);
            v.template store<R>(y + row * C, c, C);
        }
    }
}

// Each workgroup walks rows blockIdx * ROWS + group, + gridDim * ROWS, ..., and writes its
// column sums as row blockIdx of part [gridDim, 2, C], weight's and bias's.  16381 x 2048
// bfloat16: 36 us, 5.5 TB/s; 65536 x 64 float32: 11.3 us, 4.5 TB/s.
template <typename T, int LPR, int NV, Reach R>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(const T *__restrict__ grad, const T *__restrict__ x,
                                                            const T *__restrict__ weight, const float *__restrict__ mean,
                                                            const float *__restrict__ rstd, T *__restrict__ grad_x,
                                                            float *__restrict__ part, int64_t rows, int C,
                                                            int64_t x_stride, int64_t g_stride) {
    constexpr int V = kVec<T>, ROWS = kThreads / LPR;
    __shared__ float red[4];
    __shared__ float cols[ROWS > 1 ? kThreads * V : 1];
    const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
    Raw<T, V> w[NV];
    float sw[NV][V] = {}, sb[NV][V] = {};
#pragma unroll
    for (int k = 0; k < NV; ++k) w[k].template load<R>(weight, (k * LPR + lane) * V, C, true);
    const float inv = 1.f / (float)C;
    for (int64_t first = (int64_t)blockIdx.x * ROWS; first < rows; first += (int64_t)gridDim.x * ROWS) {
        const int64_t row = first + group;
        const bool on = row < rows;
        const T *xr = x + (on ? row : 0) * x_stride, *gr = grad + (on ? row : 0) * g_stride;
        const float mu = on ? mean[row] : 0.f, rs = on ? rstd[row] : 0.f;
        Raw<T, V> xv[NV], gv[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            xv[k].template load<R>(xr, (k * LPR + lane) * V, C, on);
            gv[k].template load<R>(gr, (k * LPR + lane) * V, C, on);
        }
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float xh = (xv[k][e] - mu) * rs, gw = gv[k][e] * w[k][e];  // g is zero past the row's end
                s1 += gw;
                s2 += gw * xh;
                sw[k][e] += gv[k][e] * xh;
                sb[k][e] += gv[k][e];
            }
        }
        s1 = group_sum<LPR>(s1, red) * inv;
        s2 = group_sum<LPR>(s2, red) * inv;
        if (on) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * LPR + lane) * V;
                if (c >= C) continue;
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = rs * (gv[k][e] * w[k][e] - s1 - (xv[k][e] - mu) * rs * s2);
                xv[k].set(o);
                xv[k].template store<R>(grad_x + row * C, c, C);
            }
        }
    }
    float *pw = part + (int64_t)blockIdx.x * 2 * C, *pb = pw + C;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float (&s)[V] = h == 0 ? sw[k] : sb[k];
            const int c = (k * LPR + lane) * V;
            if constexpr (ROWS > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < V; ++e) cols[threadIdx.x * V + e] = s[e];
                __syncthreads();
                for (int i = threadIdx.x; i < LPR * V; i += kThreads) {
                    float t = 0.f;
                    for (int r = 0; r < ROWS; ++r) t += cols[r * LPR * V + i];
                    if (k * LPR * V + i < C) (h == 0 ? pw : pb)[k * LPR * V + i] = t;
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (c + e < C) (h == 0 ? pw : pb)[c + e] = s[e];
            }
        }
    }
}

// Rows longer than the registers hold: grad_x from two passes over the row, one
// workgroup a row; the column sums from a second kernel, a thread a column.
template <typename T, Reach R>
__global__ __launch_bounds__(kThreads) void norm_bwd_long_kernel(const T *__restrict__ grad, const T *__restrict__ x,
                                                                 const T *__restrict__ weight,
                                                                 const float *__restrict__ mean,
                                                                 const float *__restrict__ rstd, T *__restrict__ grad_x,
                                                                 int64_t rows, int C, int64_t x_stride, int64_t g_stride) {
    constexpr int V = kVec<T>;
    __shared__ float red[4];
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T *xr = x + row * x_stride, *gr = grad + row * g_stride;
        const float mu = mean[row], rs = rstd[row];
        float s1 = 0.f, s2 = 0.f, o[V];
        Raw<T, V> xv, gv, w;
        for (int c = threadIdx.x * V; c < C; c += kThreads * V) {
            xv.template load<R>(xr, c, C, true);
            gv.template load<R>(gr, c, C, true);
            w.template load<R>(weight, c, C, true);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s1 += gv[e] * w[e];
                s2 += gv[e] * w[e] * (xv[e] - mu) * rs;
            }
        }
        s1 = group_sum<kThreads>(s1, red) / (float)C;
        s2 = group_sum<kThreads>(s2, red) / (float)C;
        for (int c = threadIdx.x * V; c < C; c += kThreads * V) {
            xv.template load<R>(xr, c, C, true);
            gv.template load<R>(gr, c, C, true);
            w.template load<R>(weight, c, C, true);
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = rs * (gv[e] * w[e] - s1 - (xv[e] - mu) * rs * s2);
            xv.set(o);
            xv.template store<R>(grad_x + row * C, c, C);
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void norm_cols_kernel(const T *__restrict__ grad, const T *__restrict__ x,
                                                             const float *__restrict__ mean,
                                                             const float *__restrict__ rstd, float *__restrict__ part,
                                                             int64_t rows, int C, int64_t x_stride, int64_t g_stride) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= C) return;
    float sw = 0.f, sb = 0.f;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const float g = Elem<T>::to_f32(grad[row * g_stride + c]);
        sw += g * (Elem<T>::to_f32(x[row * x_stride + c]) - mean[row]) * rstd[row];
        sb += g;
    }
    part[(int64_t)blockIdx.y * 2 * C + c] = sw;
    part[(int64_t)blockIdx.y * 2 * C + C + c] = sb;
}

// out0[m] (m < M0) and out1[m - M0] = sum over s, in a fixed order, of part[s][m].  64
// columns a workgroup; its 16 waves take every 16th row and are joined in LDS (512 rows of 4096:
// 4.6 us).
template <typename T>
__global__ __launch_bounds__(1024) void sum_rows_kernel(const float *__restrict__ part, int S, int64_t M0, int64_t M1,
                                                        T *__restrict__ out0, T *__restrict__ out1) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
    const int64_t M = M0 + M1, m = (int64_t)blockIdx.x * 64 + lane;
    float t = 0.f;
    if (m < M) {
        const float *p = part + m;
        int s = w;
        for (; s + 16 * 7 < S; s += 16 * 8) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = p[(int64_t)(s + 16 * e) * M];
#pragma unroll
            for (int e = 0; e < 8; ++e) t += v[e];
        }
        for (; s < S; s += 16) t += p[(int64_t)s * M];
    }
    red[w][lane] = t;
    __syncthreads();
    if (w == 0 && m < M) {
#pragma unroll
        for (int e = 1; e < 16; ++e) t += red[e][lane];
        if (m < M0) out0[m] = Elem<T>::from_f32(t);
        else out1[m - M0] = Elem<T>::from_f32(t);
    }
}

hipError_t launch_sum_rows(const float *part, int S, int64_t M0, int64_t M1, void *out0, void *out1, bool bf16,
                           hipStream_t stream) {
    const int64_t blocks = (M0 + M1 + 63) / 64;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    if (bf16)
        hipLaunchKernelGGL((sum_rows_kernel<bf16_t>), dim3((unsigned)blocks), dim3(1024), 0, stream, part, S, M0, M1,
                           (bf16_t *)out0, (bf16_t *)out1);
    else
        hipLaunchKernelGGL((sum_rows_kernel<float>), dim3((unsigned)blocks), dim3(1024), 0, stream, part, S, M0, M1,
                           (float *)out0, (float *)out1);
    return hipGetLastError();
}

namespace {

// The lanes of a row's group and the vectors each holds: the narrowest group that needs
// at most NV vectors a lane (few lanes: no idle ones in short rows and several rows a
// wave; a whole wave up to 4 vectors; the workgroup, joined through LDS, beyond it).
struct Shape {
    int lanes, nv;
};
template <typename T>
Shape shape_of(int64_t C) {
    const int64_t n = (C + kVec<T> - 1) / kVec<T>;
    if (n <= 16) return {16, 1};
    if (n <= 64) return {64, 1};
    if (n <= 128) return {64, 2};
    if (n <= 256) return {64, 4};
    if (n <= 512) return {256, 2};
    if (n <= 1024) return {256, 4};
    if (n <= 2048) return {256, 8};
    return {0, 0};
}

#define DDPM_SEQ_NORM_SHAPES(X) X(16, 1) X(64, 1) X(64, 2) X(64, 4) X(256, 2) X(256, 4) X(256, 8)

template <typename T, Reach R>
hipError_t norm_fwd(const void *x, const void *weight, const void *bias, void *y, float *mean, float *rstd, int64_t rows,
                    int64_t C, int64_t x_stride, float eps, hipStream_t stream) {
    const Shape s = shape_of<T>(C);
    const int64_t blocks = s.lanes ? (rows + kThreads / s.lanes - 1) / (kThreads / s.lanes) : (rows < 4096 ? rows : 4096);
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
#define X(L, NV)                                                                                                      \
    if (s.lanes == L && s.nv == NV)                                                                                   \
        hipLaunchKernelGGL((norm_fwd_kernel<T, L, NV, R>), dim3((unsigned)blocks), dim3(kThreads), 0, stream,         \
                           (const T *)x, (const T *)weight, (const T *)bias, (T *)y, mean, rstd, rows, (int)C,        \
                           x_stride, eps);
    if constexpr (R == kShort) {
        X(16, 1)
    } else {
        DDPM_SEQ_NORM_SHAPES(X)
        if (!s.lanes)
            hipLaunchKernelGGL((norm_fwd_long_kernel<T, R>), dim3((unsigned)blocks), dim3(kThreads), 0, stream,
                               (const T *)x, (const T *)weight, (const T *)bias, (T *)y, mean, rstd, rows, (int)C,
                               x_stride, eps);
    }
#undef X
    return hipGetLastError();
}

template <typename T, Reach R>
hipError_t norm_bwd(const void *grad, const void *x, const void *weight, const float *mean, const float *rstd,
                    void *grad_x, void *grad_weight, void *grad_bias, float *part, int64_t rows, int64_t C,
                    int64_t x_stride, int64_t g_stride, hipStream_t stream) {
    const Shape s = shape_of<T>(C);
    const int S = norm_partials(rows, C, Elem<T>::is_bf16);
#define X(L, NV)                                                                                                      \
    if (s.lanes == L && s.nv == NV)                                                                                   \
        hipLaunchKernelGGL((norm_bwd_kernel<T, L, NV, R>), dim3(S), dim3(kThreads), 0, stream, (const T *)grad,       \
                           (const T *)x, (const T *)weight, mean, rstd, (T *)grad_x, part, rows, (int)C, x_stride,    \
                           g_stride);
    if constexpr (R == kShort) {
        X(16, 1)
    } else {
        DDPM_SEQ_NORM_SHAPES(X)
        if (!s.lanes) {
            hipLaunchKernelGGL((norm_bwd_long_kernel<T, R>), dim3((unsigned)(rows < 4096 ? rows : 4096)), dim3(kThreads),
                               0, stream, (const T *)grad, (const T *)x, (const T *)weight, mean, rstd, (T *)grad_x,
                               rows, (int)C, x_stride, g_stride);
            hipLaunchKernelGGL((norm_cols_kernel<T>), dim3((unsigned)((C + kThreads - 1) / kThreads), S), dim3(kThreads),
                               0, stream, (const T *)grad, (const T *)x, mean, rstd, part, rows, (int)C, x_stride,
                               g_stride);
        }
    }
#undef X
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return launch_sum_rows(part, S, C, C, grad_weight, grad_bias, Elem<T>::is_bf16, stream);
}

#define DDPM_SEQ_NORM_REACH(T, C, CALL)                   \
    const Reach r = reach_of(C, kVec<T>);                 \
    if (r == kWhole) return CALL(kWhole);                 \
    return r == kOdd ? CALL(kOdd) : CALL(kShort);

template <typename T>
hipError_t norm_fwd(const void *x, const void *weight, const void *bias, void *y, float *mean, float *rstd, int64_t rows,
                    int64_t C, int64_t x_stride, float eps, hipStream_t stream) {
#define CALL(R) norm_fwd<T, R>(x, weight, bias, y, mean, rstd, rows, C, x_stride, eps, stream)
    DDPM_SEQ_NORM_REACH(T, C, CALL)
#undef CALL
}

template <typename T>
hipError_t norm_bwd(const void *grad, const void *x, const void *weight, const float *mean, const float *rstd,
                    void *grad_x, void *grad_weight, void *grad_bias, float *part, int64_t rows, int64_t C,
                    int64_t x_stride, int64_t g_stride, hipStream_t stream) {
#define CALL(R) \
    norm_bwd<T, R>(grad, x, weight, mean, rstd, grad_x, grad_weight, grad_bias, part, rows, C, x_stride, g_stride, stream)
    DDPM_SEQ_NORM_REACH(T, C, CALL)
#undef CALL
}

}  // namespace

int norm_partials(int64_t rows, int64_t C, bool bf16) {
    const Shape s = bf16 ? shape_of<bf16_t>(C) : shape_of<float>(C);
    const int64_t groups = s.lanes ? (rows + kThreads / s.lanes - 1) / (kThreads / s.lanes) : rows;
    const int64_t most = s.lanes ? 512 : 64;
    return (int)(groups < most ? groups : most);
}

hipError_t launch_norm_fwd(const void *x, const void *weight, const void *bias, void *y, float *mean, float *rstd,
                           int64_t rows, int64_t C, int64_t x_stride, float eps, bool bf16, hipStream_t stream) {
    return bf16 ? norm_fwd<bf16_t>(x, weight, bias, y, mean, rstd, rows, C, x_stride, eps, stream)
                : norm_fwd<float>(x, weight, bias, y, mean, rstd, rows, C, x_stride, eps, stream);
}

hipError_t launch_norm_bwd(const void *grad, const void *x, const void *weight, const float *mean, const float *rstd,
                           void *grad_x, void *grad_weight, void *grad_bias, float *part, int64_t rows, int64_t C,
                           int64_t x_stride, int64_t g_stride, bool bf16, hipStream_t stream) {
    return bf16 ? norm_bwd<bf16_t>(grad, x, weight, mean, rstd, grad_x, grad_weight, grad_bias, part, rows, C, x_stride,
                                   g_stride, stream)
                : norm_bwd<float>(grad, x, weight, mean, rstd, grad_x, grad_weight, grad_bias, part, rows, C, x_stride,
                                  g_stride, stream);
}

}  // namespace seq
}  // namespace ddpm
