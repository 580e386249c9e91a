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

// acc += sum_t w[t] X[t][p] Y[t][n] over the first n tokens of the tiles, 16 rows p by all n, as
// D[n][p].  The state is summed over the whole sequence, so it keeps float32's precision: X * w
// enters the bfloat16 products as three terms (Y is bfloat16 already).
template <typename T, int NP, int LDP, int LDN>
__device__ __forceinline__ void add_state(const T *xtile, const T *ytile, const float *w, int n, int p, int l16, int g,
                                          f32x4 (&acc)[NP / 16]) {
    for (int r = 0; r < n; r += 32) {
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
}

// What weighs a token's part in the state behind its chunk: exp(s_end - s) dt, or exp(s) in the
// adjoint before it.  Asked for an item ahead, like the tiles.
struct TimesFetch {
    float hi, lo, end_hi, end_lo, dt;
    __device__ __forceinline__ void fetch(const ScanDims &d, int64_t first, int Q, bool reverse, int tid) {
        if (tid >= Q) return;
        hi = d.shi[first + tid];
        lo = d.slo[first + tid];
        if (reverse) return;
        end_hi = d.shi[first + Q - 1];
        end_lo = d.slo[first + Q - 1];
        dt = d.dt[first + tid];
    }
    __device__ __forceinline__ void put(float *w, int Q, bool reverse, int tid) const {
        if (tid >= Q) return;
        w[tid] = reverse ? __builtin_amdgcn_exp2f(hi + lo) : __builtin_amdgcn_exp2f((end_hi - hi) + (end_lo - lo)) * dt;
    }
};

// Every chunk's own part of the state (reverse: of the adjoint), a wave 16 rows of it.  Bound by
// memory and its latency: 2 x 8192 tokens bfloat16, 32 heads, P = N = 64: 32 us, 4.2 TB/s.
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
    int id = (int)block_in_stretch();
    const int split = id % a.plan.splits;
    id /= a.plan.splits;
    const int grp = id % d.G;
    id /= d.G;
    const int c = id % d.nc, b = id / d.nc;
    const int n = valid_tokens(d.lengths, b, d.L) - c * Q;  // tokens of this chunk that count, up to Q
    if (n <= 0) return;
    const int hg = d.H / d.G, h0 = grp * hg + split * a.plan.per;
    const int h1 = h0 + a.plan.per < (grp + 1) * hg ? h0 + a.plan.per : (grp + 1) * hg;
    const int slabs = (d.P + kSlab - 1) / kSlab, items = (h1 - h0) * slabs, cols = state_cols(d.N);
    const T *xb = X + b * a.x_batch + (int64_t)c * Q * a.x_token;
    TileFetch<T, Q, NP, kThreads, false> yf;
    TileFetch<T, Q, kSlab, kThreads, WHOLE> xf;
    TimesFetch tf;
    auto chunk_of = [&](int it) { return ((int64_t)b * d.H + h0 + it / slabs) * d.nc + c; };
    auto fetch = [&](int it) {
        const int p0 = it % slabs * kSlab;
        tf.fetch(d, chunk_of(it) * Q, Q, a.reverse, tid);
        xf.fetch(xb + (int64_t)(h0 + it / slabs) * d.P + p0, a.x_token, n, d.P - p0, tid);
    };
    yf.fetch(Y + b * a.y_batch + (int64_t)c * Q * a.y_token + grp * d.N, a.y_token, n, d.N, tid);
    fetch(0);
    yf.put(ytile, LDN, n, d.N, tid);
    for (int it = 0; it < items; ++it) {
        const int p0 = it % slabs * kSlab, p = 16 * wave;
        __syncthreads();
        xf.put(xtile, LDP, n, d.P - p0, tid);
        tf.put(w, Q, a.reverse, tid);
        __syncthreads();
        if (it + 1 < items) fetch(it + 1);
        if (p0 + p >= d.P) continue;
        f32x4 acc[NP / 16];
#pragma unroll
        for (int k = 0; k < NP / 16; ++k) acc[k] = f32x4{0.f, 0.f, 0.f, 0.f};
        add_state<T, NP, LDP, LDN>(xtile, ytile, w, n < Q ? n : Q, p, l16, g, acc);
        if (p0 + p + l16 < d.P) {
            float *o = out + (chunk_of(it) * d.P + p0 + p + l16) * cols;
#pragma unroll
            for (int k = 0; k < NP / 16; ++k)
                if (16 * k + 4 * g < cols) *(f32x4 *)(o + 16 * k + 4 * g) = acc[k];
        }
    }
}

// The same for a segment of d.seg chunks, for calls that keep nothing: the running state that
// enters each chunk after the segment's first, from zero at the segment's start, the factor that a
// state at the segment's start has there, and in the place of the first chunk the state behind the
// segment, with the segment's decay.  HW heads (or slabs of them) at once share the chunk's Y and
// stay in registers over the segment.  WHOLE: P and N are in whole vectors.  Bound by the chain of
// chunks, its vector instructions (the three terms) and memory: ragged prompts 4 x 4096 bfloat16,
// 32 heads, P = 64, N = 128: 54 us.
template <typename T, int NP, bool WHOLE, int HW>
__global__ __launch_bounds__(kThreads, 2) void scan_segments_kernel(StateArgs a, const T *__restrict__ X,
                                                                 const T *__restrict__ Y, float *__restrict__ out,
                                                                 float *__restrict__ carried,
                                                                 float *__restrict__ decays) {
    constexpr int Q = 16 * kStrips<T>, LDN = NP + kVec<T>, LDP = kSlab + kVec<T>;
    __shared__ __align__(16) T ytile[Q * LDN];
    __shared__ __align__(16) T xtile[Q * LDP];
    __shared__ __align__(16) float w[Q];
    const ScanDims &d = a.d;
    const int tid = threadIdx.x, lane = tid % kWave, wave = wave_of(tid), l16 = lane % 16, g = lane / 16;
    const int nseg = (d.nc + d.seg - 1) / d.seg;
    int id = (int)block_in_stretch();
    const int split = id % a.plan.splits;
    id /= a.plan.splits;
    const int grp = id % d.G;
    id /= d.G;
    const int seg = id % nseg, b = id / nseg;
    const int len = valid_tokens(d.lengths, b, d.L), c0 = seg * d.seg, nc = (len + Q - 1) / Q;
    const int c1 = c0 + d.seg < nc ? c0 + d.seg : nc;
    if (c0 >= c1) return;
    const int slabs = (d.P + kSlab - 1) / kSlab, all = d.H / d.G * slabs, cols = state_cols(d.N), p = 16 * wave;
    // items past the group's last repeat it (and store nothing)
    auto item = [&](int i) { return split * HW + i < all ? split * HW + i : all - 1; };
    auto head = [&](int i) { return (int64_t)b * d.H + grp * (d.H / d.G) + item(i) / slabs; };
    TileFetch<T, Q, NP, kThreads, WHOLE> yf;
    TileFetch<T, Q, kSlab, kThreads, WHOLE> xf;
    TimesFetch tf;
    float decay = 1.f;
    auto fetch = [&](int c, int i) {
        const int tid = afresh(threadIdx.x), p0 = item(i) % slabs * kSlab, h = grp * (d.H / d.G) + item(i) / slabs;
        decay = d.decay[head(i) * d.nc + c];
        tf.fetch(d, (head(i) * d.nc + c) * Q, Q, false, tid);
        xf.fetch(X + b * a.x_batch + (int64_t)c * Q * a.x_token + (int64_t)h * d.P + p0, a.x_token, len - c * Q, d.P - p0, tid);
    };
    auto fetch_y = [&](int c) {
        const int tid = afresh(threadIdx.x);
        yf.fetch(Y + b * a.y_batch + (int64_t)c * Q * a.y_token + grp * d.N, a.y_token, len - c * Q, d.N, tid);
    };
    f32x4 acc[HW][NP / 16];
    float factor[HW];
    auto put = [&](int i, int c, int row) {
        float *o = out + ((head(i) * d.nc + c) * d.P + row) * cols;
#pragma unroll
        for (int k = 0; k < NP / 16; ++k)
            if (16 * k + 4 * g < cols) *(f32x4 *)(o + 16 * k + 4 * g) = acc[i][k];
    };
#pragma unroll
    for (int i = 0; i < HW; ++i) {
        factor[i] = 1.f;
#pragma unroll
        for (int k = 0; k < NP / 16; ++k) acc[i][k] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    fetch_y(c0);
    fetch(c0, 0);
    for (int c = c0; c < c1; ++c) {
        const int n = len - c * Q < Q ? len - c * Q : Q;
#pragma unroll
        for (int i = 0; i < HW; ++i) {
            const int p0 = item(i) % slabs * kSlab, row = p0 + p + l16;
            const bool mine = split * HW + i < all && row < d.P;
            __syncthreads();
            if (i == 0) yf.put(ytile, LDN, n, d.N, tid);
            xf.put(xtile, LDP, n, d.P - p0, tid);
            tf.put(w, Q, false, tid);
            const float a_c = decay;
            __syncthreads();
            if (i == 0 && c + 1 < c1) fetch_y(c + 1);
            if (i + 1 < HW) fetch(c, i + 1);
            else if (c + 1 < c1) fetch(c + 1, 0);
            if (c > c0 && mine) put(i, c, row);
            if (tid == 0 && p0 == 0 && mine) carried[head(i) * d.nc + c] = factor[i];
            factor[i] *= a_c;
#pragma unroll
            for (int k = 0; k < NP / 16; ++k) acc[i][k] *= a_c;
            add_state<T, NP, LDP, LDN>(xtile, ytile, w, n, p, l16, g, acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < HW; ++i) {
        const int row = item(i) % slabs * kSlab + p + l16;
        if (split * HW + i >= all || row >= d.P) continue;
        if (row == 0) decays[head(i) * nseg + seg] = factor[i];
        put(i, c0, row);
    }
}

// h = first; for every chunk in order: part = states[c], states[c] = h, h = decay[c] h + part.
// `rows` states a head: the chunks, or segments of d.seg of them, whose states lie d.seg apart.
// LANES of four elements by PARTS runs of states: each run goes from zero, the runs' ends are
// joined in LDS, and each run goes again from its true start; the parts stay in registers
// between where a run has at most KEEP of them and are read again otherwise.  PARTS = 1: one
// run, whose states are all in registers.  Bound by memory: 64 chunks of 2 x 32 heads, P = N = 64:
// 27 us, 5.0 TB/s; 4 segments of 4 x 32 heads, N = 128, ragged: 12 us (as 16 runs 33 us).
template <int PARTS, int LANES, int KEEP>
__global__ __launch_bounds__(PARTS *LANES) void scan_pass_kernel(ScanDims d, int Q, int rows,
                                                                 const float *__restrict__ decays,
                                                                 float *__restrict__ states,
                                                                 const float *__restrict__ first,
                                                                 float *__restrict__ final_state, int groups,
                                                                 int reverse) {
    __shared__ f32x4 ends[PARTS > 1 ? PARTS : 1][PARTS > 1 ? LANES : 1];
    __shared__ float mults[PARTS];
    const int lane = threadIdx.x % LANES, part = threadIdx.x / LANES;
    const int64_t head = blockIdx.x / groups;  // b * H + h
    const int cols = state_cols(d.N), per_row = cols / 4;
    const int e = blockIdx.x % groups * LANES + lane;  // in vectors of four
    const int64_t E = (int64_t)d.P * cols;
    const bool on = e < d.P * per_row;
    const int n = valid_tokens(d.lengths, (int)(head / d.H), d.L), nc = (n + Q * d.seg - 1) / (Q * d.seg);
    const int per = (nc + PARTS - 1) / PARTS;
    const int from = part * per < nc ? part * per : nc, to = from + per < nc ? from + per : nc;
    // where the caller's unpadded states have these four
    const int64_t user = head * d.P * d.N + (int64_t)(e / per_row) * d.N + e % per_row * 4;
    const int left = on ? d.N - e % per_row * 4 : 0;
    f32x4 *st = (f32x4 *)(states + head * d.nc * E) + (on ? e : 0);
    const float *decay = decays + head * rows;
    const int64_t each = E / 4 * d.seg, step = reverse ? -each : each;
    const int dir = reverse ? -1 : 1, c0 = reverse ? nc - 1 - from : from;
    f32x4 keep[KEEP];
    f32x4 h = {0.f, 0.f, 0.f, 0.f};
    st += c0 * each;
    decay += c0;
    const bool kept = PARTS == 1 || per <= KEEP;
    if (kept) {
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (from + k < to) keep[k] = st[k * step];
    }
    if constexpr (PARTS > 1) {
        float m = 1.f;
        if (kept) {
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
    }
    if (!on) return;
    h = first != nullptr ? load4(first + user, left) : f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (PARTS > 1)
        for (int k = 0; k < part; ++k) h = h * mults[k] + ends[k][lane];
    if (kept) {
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
    if (part == PARTS - 1 && final_state != nullptr) store4<float>(final_state + user, h, left);
}

template <typename T>
hipError_t launch_scan_states(const ScanDims &d, const T *X, int64_t x_batch, int64_t x_token, const T *Y,
                              int64_t y_batch, int64_t y_token, float *out, bool reverse, hipStream_t stream) {
    const ChunkPlan plan = plan_heads(d.B, d.nc, d.H, d.P, d.G, 1024);
    const StateArgs a = {d, plan, x_batch, x_token, y_batch, y_token, reverse ? 1 : 0};
    const int64_t blocks = (int64_t)d.B * d.nc * d.G * plan.splits;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
#define X_(NP, WHOLE) \
    hipLaunchKernelGGL((scan_states_kernel<T, NP, WHOLE>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, a, X, Y, out);
    DDPM_SEQ_SCAN_SHAPES(T, d.N, d.P, X_)
#undef X_
    return hipGetLastError();
}

template <typename T>
hipError_t launch_scan_segments(const ScanDims &d, int hw, const T *X, int64_t x_batch, int64_t x_token, const T *Y,
                                int64_t y_batch, int64_t y_token, float *states, float *carried, float *decays,
                                hipStream_t stream) {
    const int items = d.H / d.G * ((d.P + kSlab - 1) / kSlab);
    const StateArgs a = {d, {hw, (items + hw - 1) / hw}, x_batch, x_token, y_batch, y_token, 0};
    const int64_t blocks = (int64_t)d.B * ((d.nc + d.seg - 1) / d.seg) * d.G * a.plan.splits;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
#define LAUNCH(NP, WHOLE, HW)                                                                                      \
    hipLaunchKernelGGL((scan_segments_kernel<T, NP, WHOLE, HW>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, \
                       a, X, Y, states, carried, decays)
#define X_(NP, WHOLE)                                                                    \
    if (WHOLE && d.N % kVec<T> == 0) { if (hw == 2) LAUNCH(NP, true, 2); else LAUNCH(NP, true, 1); } \
    else { if (hw == 2) LAUNCH(NP, false, 2); else LAUNCH(NP, false, 1); }
    DDPM_SEQ_SCAN_SHAPES(T, d.N, d.P, X_)
#undef LAUNCH
#undef X_
    return hipGetLastError();
}
template hipError_t launch_scan_segments<float>(const ScanDims &, int, const float *, int64_t, int64_t, const float *,
                                                int64_t, int64_t, float *, float *, float *, hipStream_t);
template hipError_t launch_scan_segments<bf16_t>(const ScanDims &, int, const bf16_t *, int64_t, int64_t, const bf16_t *,
                                                 int64_t, int64_t, float *, float *, float *, hipStream_t);
template hipError_t launch_scan_states<float>(const ScanDims &, const float *, int64_t, int64_t, const float *, int64_t,
                                              int64_t, float *, bool, hipStream_t);
template hipError_t launch_scan_states<bf16_t>(const ScanDims &, const bf16_t *, int64_t, int64_t, const bf16_t *,
                                               int64_t, int64_t, float *, bool, hipStream_t);

hipError_t launch_scan_pass(const ScanDims &d, float *states, const float *decays, const float *first, float *final_state,
                            int Q, bool reverse, hipStream_t stream) {
    const int rows = (d.nc + d.seg - 1) / d.seg, vectors = d.P * state_cols(d.N) / 4;
    // A few states: a thread takes all of them.  Very many: four times the runs, so that a run is
    // short beside a memory access (training passes in float32 with 16 and 64 runs: 224 and 231 us at
    // 256 states of 8 heads, 276 and 269 us at 1024 of 2; bfloat16, 64 states of 64 heads: 356 and 415 us).
    const int lanes = rows <= 8 ? 256 : 16, groups = (vectors + lanes - 1) / lanes;
    const int64_t blocks = (int64_t)d.B * d.H * groups;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
#define X(PARTS, LANES, KEEP)                                                                                        \
    hipLaunchKernelGGL((scan_pass_kernel<PARTS, LANES, KEEP>), dim3((unsigned)blocks), dim3(PARTS * LANES), 0, stream, \
                       d, Q, rows, decays, states, first, final_state, groups, reverse ? 1 : 0)
    if (rows <= 8) X(1, 256, 8);
    else if (rows <= 256) X(16, 16, 4);
    else X(64, 16, 4);
#undef X
    return hipGetLastError();
}

}  // namespace seq
}  // namespace ddpm
