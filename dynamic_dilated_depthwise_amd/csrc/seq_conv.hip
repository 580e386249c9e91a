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

// The taps of V channels from c on (those below D), in the last W of KW; the older are 0.
template <typename T, int KW, int V, Reach R, bool EXACT>
__device__ __forceinline__ void load_taps(const T *__restrict__ weight, int c, int D, int W, float (&w)[KW][V]) {
    const int n = D - c;
    if (EXACT && R != kShort && n >= V) {  // V * KW neighbouring elements
        Raw<T, 4> r[V * KW / 4];
#pragma unroll
        for (int k = 0; k < V * KW / 4; ++k) r[k].template load<kWhole>(weight + (int64_t)c * KW + 4 * k, 0, 4, true);
#pragma unroll
        for (int e = 0; e < V; ++e)
#pragma unroll
            for (int j = 0; j < KW; ++j) w[j][e] = r[(e * KW + j) / 4][(e * KW + j) % 4];
    } else {
#pragma unroll
        for (int j = 0; j < KW; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int i = j - (KW - W);
                w[j][e] = i >= 0 && e < n ? Elem<T>::to_f32(weight[(int64_t)(c + e) * W + i]) : 0.f;
            }
    }
}

// sigmoid by the hardware's exponential and reciprocal (an ulp each; the exponent's own
// rounding is relative to u, as are those of the sum that u is).
__device__ __forceinline__ float fast_sigmoid(float u) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * u));
}

// x of sequence b (ib: its initial state) at token t < n, zero before the state's first.  A vector
// that is not there is asked for at the bias, where a row of D channels can be read in any case.
template <typename T, int V, Reach R>
__device__ __forceinline__ Raw<T, V> token(const ConvArgs &a, const T *xb, const T *ib, int t, int n, int c) {
    Raw<T, V> r;
    const bool early = t < 0, on = t < n && (!early || (ib != nullptr && t > -a.W));
    const T *p = on ? (early ? ib + (int64_t)(a.W - 1 + t) * a.D : xb + (int64_t)t * a.x_token) : (const T *)a.bias;
    r.template load<R>(p, c, a.D, on);
    return r;
}

// A thread makes `RUN` tokens: their inputs and the W - 1 before are all asked for first.  Bound
// by memory: 2 x 8192 x 2304 bfloat16, width 4: 33.5 us, 4.5 TB/s of what it must read and write.
template <typename T, int KW, bool EXACT, int V, Reach R, int RUN>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(ConvArgs a, T *__restrict__ y, T *__restrict__ last,
                                                            int64_t walks) {
    if (EXACT) a.W = KW;
    // shared tokens from the XCD's L2: 37 -> 34 us at 2 x 8192 x 2304 bfloat16, width 4
    const int64_t id = block_in_stretch() * kThreads + threadIdx.x;
    const int runs = (a.L + RUN - 1) / RUN;
    if (id >= walks) {  // the state behind the last token: W - 1 rows a sequence
        const int64_t k = id - walks;
        const int W1 = a.W - 1;
        if (last == nullptr || k >= (int64_t)a.B * W1 * a.nvec) return;
        const int c = (int)(k % a.nvec) * V, j = (int)(k / a.nvec % W1), b = (int)(k / a.nvec / W1);  // rows may pass 2^31
        const T *ib = a.initial ? (const T *)a.initial + (int64_t)b * W1 * a.D : nullptr;
        const int n = length_of(a.lengths, b, a.L);
        token<T, V, R>(a, (const T *)a.x + b * a.x_batch, ib, n - W1 + j, n, c)
            .template store<R>(last + ((int64_t)b * W1 + j) * a.D, c, a.D);
        return;
    }
    const int c = (int)(id % a.nvec) * V;
    const int64_t rest = id / a.nvec;
    const int t0 = (int)(rest % runs) * RUN, b = (int)(rest / runs);
    const int n = length_of(a.lengths, b, a.L);
    const T *xb = (const T *)a.x + b * a.x_batch;
    const T *ib = a.initial ? (const T *)a.initial + (int64_t)b * (a.W - 1) * a.D : nullptr;
    T *yb = y + ((int64_t)b * a.L + t0) * a.D;
    Raw<T, V> in[RUN + KW - 1], bias;
    float w[KW][V];
#pragma unroll
    for (int k = 0; k < RUN + KW - 1; ++k) {
        if (k < KW - a.W) in[k].r = typename Raw<T, V>::words(0);  // older than the taps
        else in[k] = token<T, V, R>(a, xb, ib, t0 - (KW - 1) + k, n, c);
    }
    load_taps<T, KW, V, R, EXACT>((const T *)a.weight, c, a.D, a.W, w);
    bias.template load<R>((const T *)a.bias, c, a.D, true);
#pragma unroll
    for (int k = 0; k < RUN; ++k) {
        if (t0 + k >= a.L) break;
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float u = bias[e];
#pragma unroll
            for (int j = 0; j < KW; ++j) u += (EXACT || j >= KW - a.W) ? w[j][e] * in[k + j][e] : 0.f;
            o[e] = t0 + k < n ? u * fast_sigmoid(u) : 0.f;
        }
        Raw<T, V> out;
        out.set(o);
        out.template store<R>(yb + (int64_t)k * a.D, c, a.D);
    }
}

constexpr int kBwdVec = 4;    // channels of a thread where it keeps windows and sums of them (backward), or has few (step)
constexpr int kBwdBatch = 4;  // tokens that are asked for ahead of the one at work

// Workgroup: cl threads along the channels by kThreads / cl walks of a.run tokens; its sums
// over the walks go to row `split` of part [splits, D * W + D].  Bound by its vector
// instructions (43 an element, three quarters of the issue slots) and by memory: 2 x 8192 x 2304
// bfloat16, width 4: 56 us, 4.0 TB/s.
template <typename T, int KW, bool EXACT, Reach R>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(ConvArgs a, const T *__restrict__ grad, int64_t g_batch,
                                                            int64_t g_token, const T *__restrict__ grad_state,
                                                            T *__restrict__ grad_x, T *__restrict__ grad_initial,
                                                            float *__restrict__ part, int cl, int blocks_c) {
    constexpr int V = kBwdVec, U = kBwdBatch;
    if (EXACT) a.W = KW;
    __shared__ float red[kThreads * V];
    const int lane = threadIdx.x % cl, walk = threadIdx.x / cl, walks = kThreads / cl;
    const int runs = (a.L + a.run - 1) / a.run;
    const int block_c = blockIdx.x % blocks_c, split = blockIdx.x / blocks_c;
    const int c = (block_c * cl + lane) * V;
    const int64_t id = (int64_t)split * walks + walk;
    float sw[KW][V] = {}, sb[V] = {};
    if (c < a.D && id < (int64_t)a.B * runs) {
        const int t0 = (int)(id % runs) * a.run, b = (int)(id / runs);
        const int n = length_of(a.lengths, b, a.L);
        const int t1 = t0 + a.run < a.L ? t0 + a.run : a.L;
        const int W1 = a.W - 1;
        const T *xb = (const T *)a.x + b * a.x_batch;
        const T *ib = a.initial ? (const T *)a.initial + (int64_t)b * W1 * a.D : nullptr;
        const T *gb = grad + b * g_batch;
        const T *gs = grad_state ? grad_state + (int64_t)b * W1 * a.D : nullptr;
        T *gx = grad_x + (int64_t)b * a.L * a.D;
        T *gi = grad_initial ? grad_initial + (int64_t)b * W1 * a.D : nullptr;
        float w[KW][V], win[KW][V], du[KW][V] = {};
        Raw<T, V> bias, x[U], g[U];
        load_taps<T, KW, V, R, EXACT>((const T *)a.weight, c, a.D, a.W, w);
        bias.template load<R>((const T *)a.bias, c, a.D, true);
#pragma unroll
        for (int j = 1; j < KW; ++j) {
            Raw<T, V> r;
            if (j > KW - a.W) r = token<T, V, R>(a, xb, ib, t0 - KW + j, n, c);
            else r.r = typename Raw<T, V>::words(0);
#pragma unroll
            for (int e = 0; e < V; ++e) win[j][e] = r[e];
        }
        auto ask = [&](int k, int t) {  // token t into slot k
            const bool on = t < n && t < t1 + W1;
            x[k].template load<R>(on ? xb + (int64_t)t * a.x_token : (const T *)a.bias, c, a.D, on);
            g[k].template load<R>(on ? gb + (int64_t)t * g_token : (const T *)a.bias, c, a.D, on);
        };
#pragma unroll
        for (int k = 0; k < U; ++k) ask(k, t0 + k);
        for (int from = t0; from < t1 + W1; from += U) {
            // step t makes du[t] (zero past the length, as g is) and emits the gradient of x at t - W1, whose last
            // term it is
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int t = from + k, at = t - W1;
#pragma unroll
                for (int j = 0; j + 1 < KW; ++j)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        win[j][e] = EXACT || j >= KW - a.W ? win[j + 1][e] : 0.f;
                        du[j][e] = du[j + 1][e];
                    }
#pragma unroll
                for (int e = 0; e < V; ++e) win[KW - 1][e] = x[k][e];
                const Raw<T, V> gc = g[k];
                ask(k, t + U);
                float o[V];
                if (t < n) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float u = bias[e];
#pragma unroll
                        for (int j = 0; j < KW; ++j) u += w[j][e] * win[j][e];
                        const float sg = fast_sigmoid(u);
                        du[KW - 1][e] = gc[e] * (sg * (1.f + u * (1.f - sg)));
                    }
                } else {  // the taps may still reach infinities before the length
#pragma unroll
                    for (int e = 0; e < V; ++e) du[KW - 1][e] = 0.f;
                }
                if (t < t1) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
#pragma unroll
                        for (int j = 0; j < KW; ++j) sw[j][e] += du[KW - 1][e] * win[j][e];
                        sb[e] += du[KW - 1][e];
                    }
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    // du[at + k] is in slot KW - W + k, the tap that it meets W - 1 - k
                    float s = 0.f;
#pragma unroll
                    for (int q = 0; q < KW; ++q) {
                        if constexpr (EXACT) {
                            s += w[KW - 1 - q][e] * du[q][e];
                        } else {
#pragma unroll
                            for (int r = 0; r < KW; ++r)
                                if (q >= KW - a.W && r == 2 * KW - 1 - a.W - q) s += w[r][e] * du[q][e];
                        }
                    }
                    o[e] = s;
                }
                if (at >= t1 || (at < t0 && !(t0 == 0 && gi != nullptr && at >= -W1))) continue;
                if (gs != nullptr && at >= n - W1 && at < n) {
                    Raw<T, V> f;
                    f.template load<R>(gs + (int64_t)(at - (n - W1)) * a.D, c, a.D, true);
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] += f[e];
                }
                Raw<T, V> out;
                out.set(o);
                out.template store<R>(at >= 0 ? gx + (int64_t)at * a.D : gi + (int64_t)(W1 + at) * a.D, c, a.D);
            }
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
// [0, S) is a place without a sequence: y is zero and no state is touched.  Latency: 3.2 us for 64
// sequences of 2304 channels.
template <typename T, int KW, bool EXACT, Reach R>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(const T *__restrict__ x, int64_t x_stride,
                                                             const T *__restrict__ weight, const T *__restrict__ bias,
                                                             T *__restrict__ state, const int *__restrict__ slots,
                                                             T *__restrict__ y, int B, int64_t S, int D, int W,
                                                             int nvec) {
    constexpr int V = kBwdVec;
    if (EXACT) W = KW;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (id >= (int64_t)B * nvec) return;
    const int c = (int)(id % nvec) * V, b = (int)(id / nvec);
    const int64_t slot = slots != nullptr ? slots[b] : b;
    float w[KW][V], u[V];
    Raw<T, V> in[KW], out;
    in[KW - 1].template load<R>(x + b * x_stride, c, D, true);
    load_taps<T, KW, V, R, EXACT>(weight, c, D, W, w);
    out.template load<R>(bias, c, D, true);
    if (slot >= 0 && slot < S) {
        T *st = state + slot * (W - 1) * D;
#pragma unroll
        for (int j = 0; j < KW - 1; ++j)
            if (j >= KW - W) in[j].template load<R>(st + (int64_t)(j - (KW - W)) * D, c, D, true);
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] = out[e];
#pragma unroll
        for (int j = 0; j < KW; ++j) {
            if (j < KW - W) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) u[e] += w[j][e] * in[j][e];
            if (j > KW - W) in[j].template store<R>(st + (int64_t)(j - (KW - W) - 1) * D, c, D);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] *= fast_sigmoid(u[e]);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] = 0.f;
    }
    out.set(u);
    out.template store<R>(y + (int64_t)b * D, c, D);
}

namespace {

struct BwdShape {
    int run, cl;
    int64_t blocks_c, splits;
};
// A walk takes whole batches with the W - 1 tokens past its run: 32 tokens (the halo is then a
// tenth for W = 4), fewer only where too few threads would be left.  Training passes with walks of
// 32 and of 8 tokens in bfloat16, width 4: 94 and 129 us at 2 x 8192 x 2304, 25.6 and 17.5 us at
// 1 x 1500 x 1024, 24 and 13.6 us at 1 x 300 x 512.
BwdShape bwd_shape(int64_t B, int64_t L, int64_t D, int W) {
    const int64_t nvec = (D + kBwdVec - 1) / kBwdVec;
    int cl = 8;
    while (cl < 64 && cl < nvec) cl *= 2;
    int batches = 8;
    while (batches > 2 && B * (L / (kBwdBatch * batches) + 1) * nvec < (1 << 16)) batches /= 2;
    const int run = kBwdBatch * batches - (W - 1);
    const int64_t walks = B * ((L + run - 1) / run), per = kThreads / cl;
    return {run, cl, (nvec + cl - 1) / cl, (walks + per - 1) / per};
}

ConvArgs args_of(const Conv &a, int V, int run) {
    return {a.x, a.weight, a.bias, a.initial, a.lengths, a.x_batch, a.x_token, (int)a.B, (int)a.L, (int)a.D, a.W,
            (int)((a.D + V - 1) / V), run};
}

// Widths 2 to 4 have kernels of their own; 1 runs in two taps and 5 to 8 in eight, the
// older ones with zero weights and no reads.  Each by how the rows of D channels are reached.
#define DDPM_SEQ_CONV_REACH(R, W, X)     \
    if ((W) == 4) X(4, true, R)          \
    else if ((W) == 3) X(3, true, R)     \
    else if ((W) == 2) X(2, true, R)     \
    else if ((W) == 1) X(2, false, R)    \
    else X(8, false, R)
#define DDPM_SEQ_CONV_WIDTHS(W, D, V, X)                              \
    if (reach_of(D, V) == kWhole) { DDPM_SEQ_CONV_REACH(kWhole, W, X) } \
    else if (reach_of(D, V) == kOdd) { DDPM_SEQ_CONV_REACH(kOdd, W, X) } \
    else { DDPM_SEQ_CONV_REACH(kShort, W, X) }

template <typename T, int RUN>
hipError_t conv_fwd(const Conv &a, void *y, void *last, hipStream_t stream) {
    constexpr int V = kVec<T>;
    const ConvArgs k = args_of(a, V, RUN);
    const int64_t walks = a.B * ((a.L + RUN - 1) / RUN) * k.nvec;
    const int64_t items = walks + (last != nullptr ? a.B * (a.W - 1) * k.nvec : 0);
    const int64_t blocks = (items + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
#define X(KW, EX, R)                                                                                               \
    hipLaunchKernelGGL((conv_fwd_kernel<T, KW, EX, V, R, RUN>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, \
                       k, (T *)y, (T *)last, walks);
    DDPM_SEQ_CONV_WIDTHS(a.W, a.D, V, X)
#undef X
    return hipGetLastError();
}

// Eight tokens a thread (11 reads for 8 results at W = 4); two where that would leave the
// chip with fewer than eight waves a compute unit.  Eight and two: 33.5 and 38 us at 2 x 8192 x
// 2304 bfloat16, 5.7 and 4.0 us at 1 x 100 x 2304.
template <typename T>
hipError_t conv_fwd(const Conv &a, void *y, void *last, hipStream_t stream) {
    const int64_t vectors = a.B * a.L * ((a.D + kVec<T> - 1) / kVec<T>);
    return vectors / 8 >= 256 * 8 * kWave ? conv_fwd<T, 8>(a, y, last, stream) : conv_fwd<T, 2>(a, y, last, stream);
}

template <typename T>
hipError_t conv_bwd(const Conv &a, const void *grad, int64_t g_batch, int64_t g_token, const void *grad_state,
                    void *grad_x, void *grad_initial, void *grad_weight, void *grad_bias, float *part,
                    hipStream_t stream) {
    const BwdShape s = bwd_shape(a.B, a.L, a.D, a.W);
    const ConvArgs k = args_of(a, kBwdVec, s.run);
    if (s.splits * s.blocks_c > 0x7fffffff) return hipErrorInvalidConfiguration;
#define X(KW, EX, R)                                                                                              \
    hipLaunchKernelGGL((conv_bwd_kernel<T, KW, EX, R>), dim3((unsigned)(s.blocks_c * s.splits)), dim3(kThreads),  \
                       0, stream, k, (const T *)grad, g_batch, g_token, (const T *)grad_state, (T *)grad_x,           \
                       (T *)grad_initial, part, s.cl, (int)s.blocks_c);
    DDPM_SEQ_CONV_WIDTHS(a.W, a.D, kBwdVec, X)
#undef X
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return launch_sum_rows(part, (int)s.splits, a.D * a.W, a.D, grad_weight, grad_bias, Elem<T>::is_bf16, stream);
}

template <typename T>
hipError_t conv_step(const void *x, int64_t x_stride, const void *weight, const void *bias, void *state,
                     const int *slots, void *y, int64_t B, int64_t S, int64_t D, int W, hipStream_t stream) {
    const int64_t nvec = (D + kBwdVec - 1) / kBwdVec, blocks = (B * nvec + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
#define X(KW, EX, R)                                                                                              \
    hipLaunchKernelGGL((conv_step_kernel<T, KW, EX, R>), dim3((unsigned)blocks), dim3(kThreads), 0, stream,       \
                       (const T *)x, x_stride, (const T *)weight, (const T *)bias, (T *)state, slots, (T *)y, (int)B, \
                       S, (int)D, W, (int)nvec);
    DDPM_SEQ_CONV_WIDTHS(W, D, kBwdVec, X)
#undef X
    return hipGetLastError();
}

}  // namespace

int conv_partials(int64_t B, int64_t L, int64_t D, int W) { return (int)bwd_shape(B, L, D, W).splits; }

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

hipError_t launch_conv_step(const void *x, int64_t x_stride, const void *weight, const void *bias, void *state,
                            const int *slots, void *y, int64_t B, int64_t S, int64_t D, int W, bool bf16,
                            hipStream_t stream) {
    return bf16 ? conv_step<bf16_t>(x, x_stride, weight, bias, state, slots, y, B, S, D, W, stream)
                : conv_step<float>(x, x_stride, weight, bias, state, slots, y, B, S, D, W, stream);
}

}  // namespace seq
}  // namespace ddpm
