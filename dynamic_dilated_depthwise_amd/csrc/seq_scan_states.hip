// seq_scan_states.hip -- the scan's chunk states and the recurrence over the chunks
// (seq_scan.hpp has the formulas).
#include "seq_scan.hpp"

namespace ddpm {
namespace seq {

constexpr int kThreads = 256;

struct StateArgs {
    ScanDims d;
    ChunkPlan plan;
    int64_t x_batch, x_token, y_batch, y_token;
    int reverse;
};

// out[p][n] = sum_t w[t] X[t][p] Y[t][n] for a chunk of a head, w = exp(s_end - s) dt, or
// exp(s) for the adjoint.  A wave holds 16 rows p by all n.  The state is summed over the
// whole sequence, so it keeps float32's precision: X * w enters the bfloat16 products as
// three terms (Y is bfloat16 already).
template <typename T, int NP, bool WHOLE>
__global__ __launch_bounds__(kThreads) void scan_states_kernel(StateArgs a, const T *__restrict__ X,
                                                               const T *__restrict__ Y, float *__restrict__ out) {
    // 16 bytes of padding only: a workgroup more fits a compute unit, which is worth more than its bank conflicts
    constexpr int Q = 16 * kStrips<T>, LDN = NP + kVec<T>, LDP = kSlab + kVec<T>;
    __shared__ __align__(16) T ytile[Q * LDN];
    __shared__ __align__(16) T xtile[Q * LDP];
    __shared__ __align__(16) float w[Q];
    const ScanDims &d = a.d;
    const int tid = threadIdx.x, lane = tid % kWave, wave = wave_of(tid), l16 = lane % 16, g = lane / 16;
    int id = blockIdx.x;
    const int split = id % a.plan.splits;
    id /= a.plan.splits;
    const int grp = id % d.G;
    id /= d.G;
    const int c = id % d.nc, b = id / d.nc;
    const int n = valid_tokens(d.lengths, b, d.L) - c * Q;  // tokens of this chunk that count, up to Q
    if (n <= 0) return;
    const int hg = d.H / d.G, h0 = grp * hg + split * a.plan.per;
    const int h1 = h0 + a.plan.per < (grp + 1) * hg ? h0 + a.plan.per : (grp + 1) * hg;
    const int slabs = (d.P + kSlab - 1) / kSlab, items = (h1 - h0) * slabs;
    const T *xb = X + b * a.x_batch + (int64_t)c * Q * a.x_token;
    TileFetch<T, Q, NP, kThreads, false> yf;
    TileFetch<T, Q, kSlab, kThreads, WHOLE> xf;
    yf.fetch(Y + b * a.y_batch + (int64_t)c * Q * a.y_token + grp * d.N, a.y_token, n, d.N, tid);
    xf.fetch(xb + (int64_t)h0 * d.P, a.x_token, n, d.P, tid);
    yf.put(ytile, LDN, n, d.N, tid);
    for (int it = 0; it < items; ++it) {
        const int h = h0 + it / slabs, p0 = it % slabs * kSlab;
        __syncthreads();
        xf.put(xtile, LDP, n, d.P - p0, tid);
        if (tid < Q) {
            const int64_t at = ((int64_t)(b * d.H + h) * d.nc + c) * Q;
            float f = d.shi[at + tid], l = d.slo[at + tid];
            if (!a.reverse) {
                f = d.shi[at + Q - 1] - f;
                l = d.slo[at + Q - 1] - l;
            }
            w[tid] = __builtin_amdgcn_exp2f(f + l) * (a.reverse ? 1.f : d.dt[at + tid]);
        }
        __syncthreads();
        if (it + 1 < items) {
            const int hn = h0 + (it + 1) / slabs, pn = (it + 1) % slabs * kSlab;
            xf.fetch(xb + (int64_t)hn * d.P + pn, a.x_token, n, d.P - pn, tid);
        }
        const int p = 16 * wave;
        if (p0 + p >= d.P) continue;
        f32x4 acc[NP / 16];
#pragma unroll
        for (int k = 0; k < NP / 16; ++k) acc[k] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int r = 0; r < (n < Q ? n : Q); r += 32) {
            const Frag<T> xr = col_frag(xtile, LDP, r, p, l16, g);
            const f32x4 wa = *(const f32x4 *)(w + r + 4 * g), wb = *(const f32x4 *)(w + r + 16 + 4 * g);
            Frag<T> xs[kTerms<T>];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float we = e < 4 ? wa[e % 4] : wb[e % 4];
                if constexpr (Elem<T>::is_bf16) {
                    __bf16 t0, t1, t2;
                    split3((float)xr[e] * we, t0, t1, t2);
                    xs[0][e] = t0;
                    xs[1][e] = t1;
                    xs[2][e] = t2;
                } else {
                    xs[0].v[e] = xr.v[e] * we;
                }
            }
#pragma unroll
            for (int k = 0; k < NP / 16; ++k) {
                const Frag<T> yr = col_frag(ytile, LDN, r, 16 * k, l16, g);
#pragma unroll
                for (int t = 0; t < kTerms<T>; ++t) acc[k] = mma(yr, xs[t], acc[k]);
            }
        }
        if (p0 + p + l16 < d.P) {
            const int cols = state_cols(d.N);
            float *o = out + (((int64_t)(b * d.H + h) * d.nc + c) * d.P + p0 + p + l16) * cols;
#pragma unroll
            for (int k = 0; k < NP / 16; ++k)
                if (16 * k + 4 * g < cols) *(f32x4 *)(o + 16 * k + 4 * g) = acc[k];
        }
    }
}

constexpr int kPassLanes = 16;

// h = first; for every chunk in order: part = states[c], states[c] = h, h = decay[c] h + part.
// Sixteen lanes of four elements by PARTS runs of chunks: each run goes from zero, the runs'
// ends are joined in LDS, and each run goes again from its true start; the parts stay in
// registers between where a run has at most KEEP chunks and are read again otherwise.
template <int PARTS>
__global__ __launch_bounds__(PARTS *kPassLanes) void scan_pass_kernel(ScanDims d, int Q, float *__restrict__ states,
                                                                      const float *__restrict__ first,
                                                                      float *__restrict__ final_state, int groups,
                                                                      int reverse) {
    constexpr int KEEP = 4;
    __shared__ f32x4 ends[PARTS][kPassLanes];
    __shared__ float mults[PARTS];
    const int lane = threadIdx.x % kPassLanes, part = threadIdx.x / kPassLanes;
    const int64_t head = blockIdx.x / groups;  // b * H + h
    const int cols = state_cols(d.N), per_row = cols / 4;
    const int e = blockIdx.x % groups * kPassLanes + lane;  // in vectors of four
    const int64_t E = (int64_t)d.P * cols;
    const bool on = e < d.P * per_row;
    const int n = valid_tokens(d.lengths, (int)(head / d.H), d.L), nc = (n + Q - 1) / Q;
    const int per = (nc + PARTS - 1) / PARTS;
    const int from = part * per < nc ? part * per : nc, to = from + per < nc ? from + per : nc;
    // where the caller's unpadded states have these four
    const int64_t user = head * d.P * d.N + (int64_t)(e / per_row) * d.N + e % per_row * 4;
    const int left = on ? d.N - e % per_row * 4 : 0;
    f32x4 *st = (f32x4 *)(states + head * d.nc * E) + (on ? e : 0);
    const float *decay = d.decay + head * d.nc;
    const int64_t step = reverse ? -E / 4 : E / 4;
    const int dir = reverse ? -1 : 1, c0 = reverse ? nc - 1 - from : from;
    f32x4 keep[KEEP];
    f32x4 h = {0.f, 0.f, 0.f, 0.f};
    float m = 1.f;
    st += c0 * (E / 4);
    decay += c0;
    if (per <= KEEP) {
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (from + k < to) keep[k] = st[k * step];
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (from + k < to) {
                h = h * decay[k * dir] + keep[k];
                m *= decay[k * dir];
            }
    } else {
#pragma unroll 8
        for (int k = 0; k < to - from; ++k) {
            h = h * decay[k * dir] + st[k * step];
            m *= decay[k * dir];
        }
    }
    ends[part][lane] = h;
    if (lane == 0) mults[part] = m;
    __syncthreads();
    h = first != nullptr ? load4(first + user, left) : f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < part; ++k) h = h * mults[k] + ends[k][lane];
    if (part == PARTS - 1 && final_state != nullptr && on) store4<float>(final_state + user, h * mults[part] + ends[part][lane], left);
    if (!on) return;
    if (per <= KEEP) {
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (from + k < to) {
                st[k * step] = h;
                h = h * decay[k * dir] + keep[k];
            }
    } else {
#pragma unroll 8
        for (int k = 0; k < to - from; ++k) {
            const f32x4 own = st[k * step];
            st[k * step] = h;
            h = h * decay[k * dir] + own;
        }
    }
}

template <typename T>
hipError_t launch_scan_states(const ScanDims &d, const T *X, int64_t x_batch, int64_t x_token, const T *Y,
                              int64_t y_batch, int64_t y_token, float *out, bool reverse, hipStream_t stream) {
    const ChunkPlan plan = plan_heads(d.B, d.nc, d.H, d.G, 1024);
    const StateArgs a = {d, plan, x_batch, x_token, y_batch, y_token, reverse ? 1 : 0};
    const int64_t blocks = (int64_t)d.B * d.nc * d.G * plan.splits;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
#define X_(NP, WHOLE) \
    hipLaunchKernelGGL((scan_states_kernel<T, NP, WHOLE>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, a, X, Y, out);
    DDPM_SEQ_SCAN_SHAPES(T, d.N, d.P, X_)
#undef X_
    return hipGetLastError();
}
template hipError_t launch_scan_states<float>(const ScanDims &, const float *, int64_t, int64_t, const float *, int64_t,
                                              int64_t, float *, bool, hipStream_t);
template hipError_t launch_scan_states<bf16_t>(const ScanDims &, const bf16_t *, int64_t, int64_t, const bf16_t *,
                                               int64_t, int64_t, float *, bool, hipStream_t);

hipError_t launch_scan_pass(const ScanDims &d, float *states, const float *first, float *final_state, int Q,
                            bool reverse, hipStream_t stream) {
    const int groups = (d.P * state_cols(d.N) / 4 + kPassLanes - 1) / kPassLanes;
    const int64_t blocks = (int64_t)d.B * d.H * groups;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
    // many chunks: four times the runs, so that a run is short beside a memory access
    if (d.nc <= 128)
        hipLaunchKernelGGL((scan_pass_kernel<16>), dim3((unsigned)blocks), dim3(16 * kPassLanes), 0, stream, d, Q, states,
                           first, final_state, groups, reverse ? 1 : 0);
    else
        hipLaunchKernelGGL((scan_pass_kernel<64>), dim3((unsigned)blocks), dim3(64 * kPassLanes), 0, stream, d, Q, states,
                           first, final_state, groups, reverse ? 1 : 0);
    return hipGetLastError();
}

}  // namespace seq
}  // namespace ddpm
