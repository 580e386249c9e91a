// seq_conv.hip -- short causal convolution along a sequence with SiLU, channels last:
//
//   u[t, d] = bias[d] + sum_j weight[d, j] * x[t - (W - 1) + j, d],   y = u * sigmoid(u)
//
// where x before the first token is the initial state (zeros without one).  Bound by
// memory: each element is read and written once and takes a few dozen operations.  A
// thread holds 16 bytes of neighbouring channels, walks a run of tokens and keeps the
// last W - 1 inputs in registers; neighbouring threads hold neighbouring channels, so
// every access of a wave is one contiguous piece of a token's row.
//
// Backward.  With du = g * sigmoid(u) * (1 + u * (1 - sigmoid(u))) (u made again from x):
//   grad_x[t] = sum_k weight[W - 1 - k] * du[t + k]
//   grad_weight[j] = sum_t du[t] * x[t - (W - 1) + j],  grad_bias = sum_t du[t]
// The walk makes du W - 1 tokens past its run (a neighbour makes those again) and emits
// grad_x that far behind.  The column sums leave each workgroup as one float32 row.
#include "seq_common.hpp"
#include "seq_launch.hpp"

namespace ddpm {
namespace seq {

constexpr int kThreads = 256;

struct ConvArgs {
    const void *x, *weight, *bias, *initial;
    const int *lengths;
    int64_t x_batch, x_token;
    int B, L, D, W, nvec, run;
};

__device__ __forceinline__ int length_of(const int *lengths, int b, int L) {
    if (lengths == nullptr) return L;
    const int n = lengths[b];
    return n < 0 ? 0 : n > L ? L : n;
}

// The weights of V channels, tap by tap, in the last W of KW taps (the first KW - W are 0).
template <typename T, int KW>
__device__ __forceinline__ void load_taps(const T *weight, int c, int D, int W, float (&w)[KW][kVec<T>]) {
#pragma unroll
    for (int j = 0; j < KW; ++j)
#pragma unroll
        for (int e = 0; e < kVec<T>; ++e) {
            const int i = j - (KW - W);
            w[j][e] = i >= 0 && c + e < D ? Elem<T>::to_f32(weight[(int64_t)(c + e) * W + i]) : 0.f;
        }
}

// x at token t of sequence b (t < 0: the initial state's row W - 1 + t), as raw bytes.
template <typename T>
__device__ __forceinline__ u32x4 token(const ConvArgs &a, const T *xb, const T *ib, int t, int c) {
    if (t >= 0) return load_vec<T>(xb + (int64_t)t * a.x_token + c, a.D - c);
    if (ib != nullptr && t >= 1 - a.W) return load_vec<T>(ib + (int64_t)(a.W - 1 + t) * a.D + c, a.D - c);
    return u32x4{0, 0, 0, 0};
}

template <typename T, int KW, bool EXACT>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(ConvArgs a, T *__restrict__ y, T *__restrict__ last,
                                                            int64_t walks) {
    constexpr int V = kVec<T>;
    if (EXACT) a.W = KW;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int runs = (a.L + a.run - 1) / a.run;
    if (id >= walks) {  // the state behind the last token: W - 1 rows a sequence
        const int64_t k = id - walks;
        const int W1 = a.W - 1;
        if (last == nullptr || k >= (int64_t)a.B * W1 * a.nvec) return;
        const int c = (int)(k % a.nvec) * V, j = (int)(k / a.nvec) % W1, b = (int)(k / a.nvec / W1);
        const T *ib = a.initial ? (const T *)a.initial + (int64_t)b * W1 * a.D : nullptr;
        float v[V];
        widen<T>(token<T>(a, (const T *)a.x + b * a.x_batch, ib, length_of(a.lengths, b, a.L) - W1 + j, c), v);
        store_vec<T>(last + ((int64_t)b * W1 + j) * a.D + c, v, a.D - c);
        return;
    }
    const int c = (int)(id % a.nvec) * V;
    const int64_t rest = id / a.nvec;
    const int t0 = (int)(rest % runs) * a.run, b = (int)(rest / runs);
    const int n = length_of(a.lengths, b, a.L);
    const int t1 = t0 + a.run < a.L ? t0 + a.run : a.L;
    const T *xb = (const T *)a.x + b * a.x_batch;
    const T *ib = a.initial ? (const T *)a.initial + (int64_t)b * (a.W - 1) * a.D : nullptr;
    T *yb = y + (int64_t)b * a.L * a.D + c;
    float w[KW][V], bias[V], win[KW][V];
    load_taps<T, KW>((const T *)a.weight, c, a.D, a.W, w);
    widen<T>(load_vec<T>((const T *)a.bias + c, a.D - c), bias);
#pragma unroll
    for (int j = 1; j < KW; ++j)  // taps older than W - 1 read as zero: their weight is zero, x there need not be finite
        if (t0 < n && j >= KW - a.W + 1) widen<T>(token<T>(a, xb, ib, t0 - KW + j, c), win[j]);
        else
#pragma unroll
            for (int e = 0; e < V; ++e) win[j][e] = 0.f;
#pragma unroll 4
    for (int t = t0; t < t1; ++t) {
        float u[V];
        if (t < n) {
#pragma unroll
            for (int j = 0; j + 1 < KW; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e) win[j][e] = j >= KW - a.W ? win[j + 1][e] : 0.f;
            widen<T>(load_vec<T>(xb + (int64_t)t * a.x_token + c, a.D - c), win[KW - 1]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float s = bias[e];
#pragma unroll
                for (int j = 0; j < KW; ++j) s += w[j][e] * win[j][e];
                u[e] = s * sigmoid(s);
            }
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) u[e] = 0.f;
        }
        store_vec<T>(yb + (int64_t)t * a.D, u, a.D - c);
    }
}

// Workgroup: cl threads along the channels by kThreads / cl walks of a.run tokens; its sums
// over the walks go to row `split` of part [splits, D * W + D].
template <typename T, int KW, bool EXACT>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(ConvArgs a, const T *__restrict__ grad, int64_t g_batch,
                                                            int64_t g_token, const T *__restrict__ grad_state,
                                                            T *__restrict__ grad_x, T *__restrict__ grad_initial,
                                                            float *__restrict__ part, int cl, int blocks_c) {
    constexpr int V = kVec<T>;
    if (EXACT) a.W = KW;
    __shared__ float red[kThreads * V];
    const int lane = threadIdx.x % cl, walk = threadIdx.x / cl, walks = kThreads / cl;
    const int runs = (a.L + a.run - 1) / a.run;
    const int block_c = blockIdx.x % blocks_c, split = blockIdx.x / blocks_c;
    const int c = (block_c * cl + lane) * V;
    const int64_t id = (int64_t)split * walks + walk;
    float w[KW][V], bias[V], sw[KW][V] = {}, sb[V] = {};
    if (c < a.D && id < (int64_t)a.B * runs) {
        const int t0 = (int)(id % runs) * a.run, b = (int)(id / runs);
        const int n = length_of(a.lengths, b, a.L);
        const int t1 = t0 + a.run < a.L ? t0 + a.run : a.L;
        const int W1 = a.W - 1;
        const T *xb = (const T *)a.x + b * a.x_batch;
        const T *ib = a.initial ? (const T *)a.initial + (int64_t)b * W1 * a.D : nullptr;
        const T *gb = grad + b * g_batch + c;
        const T *gs = grad_state ? grad_state + (int64_t)b * W1 * a.D + c : nullptr;
        T *gx = grad_x + (int64_t)b * a.L * a.D + c;
        T *gi = grad_initial ? grad_initial + (int64_t)b * W1 * a.D + c : nullptr;
        load_taps<T, KW>((const T *)a.weight, c, a.D, a.W, w);
        widen<T>(load_vec<T>((const T *)a.bias + c, a.D - c), bias);
        float win[KW][V], du[KW][V] = {};
#pragma unroll
        for (int j = 1; j < KW; ++j)
            if (t0 < n && j >= KW - a.W + 1) widen<T>(token<T>(a, xb, ib, t0 - KW + j, c), win[j]);
            else
#pragma unroll
                for (int e = 0; e < V; ++e) win[j][e] = 0.f;
        // Step t makes du[t] and emits the gradient of x at t - W1, whose last term it is.
        for (int t = t0; t < t1 + W1; ++t) {
#pragma unroll
            for (int j = 0; j + 1 < KW; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    win[j][e] = j >= KW - a.W ? win[j + 1][e] : 0.f;
                    du[j][e] = du[j + 1][e];
                }
            if (t < n) {
                float g[V];
                widen<T>(load_vec<T>(xb + (int64_t)t * a.x_token + c, a.D - c), win[KW - 1]);
                widen<T>(load_vec<T>(gb + (int64_t)t * g_token, a.D - c), g);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float s = bias[e];
#pragma unroll
                    for (int j = 0; j < KW; ++j) s += w[j][e] * win[j][e];
                    const float sg = sigmoid(s);
                    du[KW - 1][e] = g[e] * sg * (1.f + s * (1.f - sg));
                }
                if (t < t1) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
#pragma unroll
                        for (int j = 0; j < KW; ++j) sw[j][e] += du[KW - 1][e] * win[j][e];
                        sb[e] += du[KW - 1][e];
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) du[KW - 1][e] = win[KW - 1][e] = 0.f;
            }
            const int at = t - W1;  // grad_x[at] = sum_k w[KW - 1 - k] du[at + k], du[at + k] in slot KW - W + k
            if (at < t0 && !(t0 == 0 && gi != nullptr)) continue;
            if (at >= t1) continue;
            float s[V] = {};
#pragma unroll
            for (int q = 0; q < KW; ++q) {
                // slot q holds du[t - (KW - 1) + q] = du[at + k], k = q - (KW - W); its weight's tap is W - 1 - k
                if (q >= KW - a.W) {
#pragma unroll
                    for (int r = 0; r < KW; ++r)
                        if (r == 2 * KW - 1 - a.W - q) {
#pragma unroll
                            for (int e = 0; e < V; ++e) s[e] += w[r][e] * du[q][e];
                        }
                }
            }
            if (gs != nullptr && at >= n - W1 && at < n) {
                float f[V];
                widen<T>(load_vec<T>(gs + (int64_t)(at - (n - W1)) * a.D, a.D - c), f);
#pragma unroll
                for (int e = 0; e < V; ++e) s[e] += f[e];
            }
            if (at >= 0) store_vec<T>(gx + (int64_t)at * a.D, s, a.D - c);
            else store_vec<T>(gi + (int64_t)(W1 + at) * a.D, s, a.D - c);
        }
    }
    const int64_t M = (int64_t)a.D * (a.W + 1);
    float *row = part + split * M;
#pragma unroll
    for (int j = 0; j <= KW; ++j) {
        if (j < KW - a.W) continue;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) red[threadIdx.x * V + e] = j < KW ? sw[j < KW ? j : 0][e] : sb[e];
        __syncthreads();
        for (int i = threadIdx.x; i < cl * V; i += kThreads) {
            const int64_t d = (int64_t)block_c * cl * V + i;
            if (d >= a.D) continue;
            float t = 0.f;
            for (int r = 0; r < walks; ++r) t += red[r * cl * V + i];
            if (j < KW) row[d * a.W + j - (KW - a.W)] = t;
            else row[(int64_t)a.D * a.W + d] = t;
        }
    }
}

// One token of each sequence: state rows hold the W - 1 inputs before it.  A slot outside
// [0, S) is a place without a sequence: y is zero and no state is touched.
template <typename T, int KW, bool EXACT>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(const T *__restrict__ x, int64_t x_stride,
                                                             const T *__restrict__ weight, const T *__restrict__ bias,
                                                             T *__restrict__ state, const int *__restrict__ slots,
                                                             T *__restrict__ y, int B, int64_t S, int D, int W,
                                                             int nvec) {
    constexpr int V = kVec<T>;
    if (EXACT) W = KW;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (id >= (int64_t)B * nvec) return;
    const int c = (int)(id % nvec) * V, b = (int)(id / nvec);
    const int64_t slot = slots != nullptr ? slots[b] : b;
    float u[V] = {};
    if (slot >= 0 && slot < S) {
        T *st = state + slot * (W - 1) * D + c;
        float w[KW][V], v[V];
        u32x4 in[KW];
#pragma unroll
        for (int j = 0; j < KW; ++j) {
            in[j] = u32x4{0, 0, 0, 0};
            if (j == KW - 1) in[j] = load_vec<T>(x + b * x_stride + c, D - c);
            else if (j >= KW - W) in[j] = load_vec<T>(st + (int64_t)(j - (KW - W)) * D, D - c);
        }
        load_taps<T, KW>(weight, c, D, W, w);
        widen<T>(load_vec<T>(bias + c, D - c), u);
#pragma unroll
        for (int j = 0; j < KW; ++j) {
            widen<T>(in[j], v);
#pragma unroll
            for (int e = 0; e < V; ++e) u[e] += w[j][e] * v[e];
            if (j >= KW - W + 1) store_vec<T>(st + (int64_t)(j - (KW - W) - 1) * D, v, D - c);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] *= sigmoid(u[e]);
    }
    store_vec<T>(y + (int64_t)b * D + c, u, D - c);
}

namespace {

// Tokens a thread walks: as long as at least 2^18 threads (16 waves a SIMD's worth of
// loads in flight over the chip) are left, from 1 to 32.
int run_of(int64_t B, int64_t L, int64_t nvec) {
    int run = 1;
    while (run < 32 && B * L * nvec / (2 * run) >= (1 << 18)) run *= 2;
    return run;
}

struct BwdShape {
    int run, cl;
    int64_t blocks_c, splits;
};
// The backward's halo costs W - 1 extra tokens a run and its partials one row a
// workgroup: runs of 32, shorter only where too few threads would be left.
BwdShape bwd_shape(int64_t B, int64_t L, int64_t D, bool bf16) {
    const int64_t nvec = (D * (bf16 ? 2 : 4) + 15) / 16;
    int cl = 8;
    while (cl < 32 && cl < nvec) cl *= 2;
    int run = 32;
    while (run > 4 && B * ((L + run - 1) / run) * nvec < (1 << 16)) run /= 2;
    const int64_t walks = B * ((L + run - 1) / run), per = kThreads / cl;
    return {run, cl, (nvec + cl - 1) / cl, (walks + per - 1) / per};
}

ConvArgs args_of(const Conv &a, bool bf16, int run) {
    return {a.x, a.weight, a.bias, a.initial, a.lengths, a.x_batch, a.x_token, (int)a.B, (int)a.L, (int)a.D, a.W,
            (int)((a.D * (bf16 ? 2 : 4) + 15) / 16), run};
}

// Widths 2 to 4 have kernels of their own; 1 runs in two taps and 5 to 8 in eight, the
// older ones with zero weights and no reads.
#define DDPM_SEQ_CONV_WIDTHS(X)    \
    if (a.W == 4) X(4, true)       \
    else if (a.W == 3) X(3, true)  \
    else if (a.W == 2) X(2, true)  \
    else if (a.W == 1) X(2, false) \
    else X(8, false)

template <typename T>
hipError_t conv_fwd(const Conv &a, void *y, void *last, hipStream_t stream) {
    ConvArgs k = args_of(a, Elem<T>::is_bf16, 1);
    k.run = run_of(a.B, a.L, k.nvec);
    const int64_t walks = a.B * ((a.L + k.run - 1) / k.run) * k.nvec;
    const int64_t items = walks + (last != nullptr ? a.B * (a.W - 1) * k.nvec : 0);
    const int64_t blocks = (items + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
#define X(KW, EX)                                                                                                  \
    hipLaunchKernelGGL((conv_fwd_kernel<T, KW, EX>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, k, (T *)y, \
                       (T *)last, walks);
    DDPM_SEQ_CONV_WIDTHS(X)
#undef X
    return hipGetLastError();
}

template <typename T>
hipError_t conv_bwd(const Conv &a, const void *grad, int64_t g_batch, int64_t g_token, const void *grad_state,
                    void *grad_x, void *grad_initial, void *grad_weight, void *grad_bias, float *part,
                    hipStream_t stream) {
    const BwdShape s = bwd_shape(a.B, a.L, a.D, Elem<T>::is_bf16);
    const ConvArgs k = args_of(a, Elem<T>::is_bf16, s.run);
    if (s.splits * s.blocks_c > 0x7fffffff) return hipErrorInvalidConfiguration;
#define X(KW, EX)                                                                                                         \
    hipLaunchKernelGGL((conv_bwd_kernel<T, KW, EX>), dim3((unsigned)(s.blocks_c * s.splits)), dim3(kThreads), 0,     \
                       stream, k, (const T *)grad, g_batch, g_token, (const T *)grad_state, (T *)grad_x,              \
                       (T *)grad_initial, part, s.cl, (int)s.blocks_c);
    DDPM_SEQ_CONV_WIDTHS(X)
#undef X
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return launch_sum_rows(part, (int)s.splits, a.D * a.W, a.D, grad_weight, grad_bias, Elem<T>::is_bf16, stream);
}

}  // namespace

int conv_partials(int64_t B, int64_t L, int64_t D, bool bf16) { return (int)bwd_shape(B, L, D, bf16).splits; }

hipError_t launch_conv_fwd(const Conv &a, void *y, void *last, bool bf16, hipStream_t stream) {
    return bf16 ? conv_fwd<bf16_t>(a, y, last, stream) : conv_fwd<float>(a, y, last, stream);
}

hipError_t launch_conv_bwd(const Conv &a, const void *grad, int64_t g_batch, int64_t g_token, const void *grad_state,
                           void *grad_x, void *grad_initial, void *grad_weight, void *grad_bias, float *part, bool bf16,
                           hipStream_t stream) {
    return bf16 ? conv_bwd<bf16_t>(a, grad, g_batch, g_token, grad_state, grad_x, grad_initial, grad_weight, grad_bias,
                                   part, stream)
                : conv_bwd<float>(a, grad, g_batch, g_token, grad_state, grad_x, grad_initial, grad_weight, grad_bias,
                                  part, stream);
}

template <typename T>
static hipError_t conv_step(const void *x, int64_t x_stride, const void *weight, const void *bias, void *state,
                            const int *slots, void *y, int64_t B, int64_t S, int64_t D, int W, hipStream_t stream) {
    const int64_t nvec = (D + kVec<T> - 1) / kVec<T>, blocks = (B * nvec + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    struct {
        int W;
    } a = {W};
#define X(KW, EX)                                                                                                          \
    hipLaunchKernelGGL((conv_step_kernel<T, KW, EX>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, (const T *)x,     \
                       x_stride, (const T *)weight, (const T *)bias, (T *)state, slots, (T *)y, (int)B, S, (int)D, W,  \
                       (int)nvec);
    DDPM_SEQ_CONV_WIDTHS(X)
#undef X
    return hipGetLastError();
}

hipError_t launch_conv_step(const void *x, int64_t x_stride, const void *weight, const void *bias, void *state,
                            const int *slots, void *y, int64_t B, int64_t S, int64_t D, int W, bool bf16,
                            hipStream_t stream) {
    return bf16 ? conv_step<bf16_t>(x, x_stride, weight, bias, state, slots, y, B, S, D, W, stream)
                : conv_step<float>(x, x_stride, weight, bias, state, slots, y, B, S, D, W, stream);
}

}  // namespace seq
}  // namespace ddpm
