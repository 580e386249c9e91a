// seq_scan_fwd.hip -- the selective scan over whole sequences: times and outputs of the
// chunks (seq_scan.hpp has the formulas), and the single-token step.
#include "seq_scan.hpp"

namespace ddpm {
namespace seq {

constexpr int kThreads = 256;
constexpr int kTimeHeads = 4;
constexpr double kLog2e = 1.4426950408889634;

// dt and the running sums s of a chunk, four heads a workgroup (dt's rows lie token by
// token in memory, what comes out head by head), a wave a head, 64-bit sums.  A token past
// the sequence's length has dt = 0 and no decay: it leaves the state alone.  A step's decay is bounded
// to 2^-2000 and 2^2000, beyond which float32 has only 0 and infinity, so that s stays
// finite.  2 x 8192 tokens, 32 heads: 6.7 us, most of it latency.
template <typename T>
__global__ __launch_bounds__(kThreads) void scan_times_kernel(ScanDims d, const T *__restrict__ raw, int64_t batch,
                                                              int64_t token, const float *__restrict__ A,
                                                              const float *__restrict__ bias, int blocks_h) {
    constexpr int Q = 16 * kStrips<T>, PER = Q / kWave;
    __shared__ float tile[kTimeHeads][Q + 1];
    const int h0 = blockIdx.x % blocks_h * kTimeHeads, c = blockIdx.x / blocks_h % d.nc, b = blockIdx.x / blocks_h / d.nc;
    const int n = valid_tokens(d.lengths, b, d.L) - c * Q;
    for (int i = threadIdx.x; i < Q * kTimeHeads; i += kThreads) {
        const int t = i / kTimeHeads, h = h0 + i % kTimeHeads;
        float v = 0.f;
        if (t < n && h < d.H) v = softplus(Elem<T>::to_f32(raw[b * batch + (int64_t)(c * Q + t) * token + h]) + bias[h]);
        tile[i % kTimeHeads][t] = v;
    }
    __syncthreads();
    const int lane = threadIdx.x % kWave;
    const int k = threadIdx.x / kWave;
    if (h0 + k < d.H) {
        const double a = A[h0 + k] * kLog2e;
        const int64_t at = (((int64_t)b * d.H + h0 + k) * d.nc + c) * Q + lane * PER;
        double s[PER], run = 0.;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const float v = tile[k][lane * PER + e];
            d.dt[at + e] = v;
            const double step = v * a;
            run += lane * PER + e >= n ? 0. : step < -2000. ? -2000. : step > 2000. ? 2000. : step;  // NaN stays NaN
            s[e] = run;
        }
        double all = run;
#pragma unroll
        for (int m = 1; m < kWave; m *= 2) {
            const double o = __shfl_up(all, m, kWave);
            if (lane >= m) all += o;
        }
        double before = __shfl_up(all, 1, kWave);  // not all - run: NaN must reach no earlier token
        if (lane == 0) before = 0.;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const float hi = (float)(before + s[e]);
            d.shi[at + e] = hi;
            d.slo[at + e] = (float)(before + s[e] - hi);
        }
        if (lane == kWave - 1)
            d.decay[((int64_t)b * d.H + h0 + k) * d.nc + c] = __builtin_amdgcn_exp2f((float)all);
    }
}

struct OutArgs {
    ScanDims d;
    ChunkPlan plan;
    int64_t x_batch, x_token, b_batch, b_token, c_batch, c_token;
    const float *states;   // [B, H, nc, P, cols]: the state that enters each chunk; with segments that of a
                           // segment at its first, and at the others what the segment's own tokens add to it there
    const float *carried;  // [B, H, nc]: the factor of the segment's state at a chunk of it
    int has_first;         // an initial state
    const float *D;
};

// One row of the state over the n tokens of a chunk, in four threads, from what enters it in v (a
// quarter of the columns in each): the y that are not finite become the recurrence's.
template <typename T, int NP>
__device__ __forceinline__ void recur(const ScanDims &d, int64_t head, int c, int n, bool mine, float (&v)[NP / 4],
                                      const T *x, int64_t x_token, const T *B, int64_t b_token, const T *C,
                                      int64_t c_token, float skip, T *y) {
    const int64_t at = (head * d.nc + c) * (16 * kStrips<T>);
    float hi = 0.f, lo = 0.f;
    for (int t = 0; t < n; ++t) {
        const float next_hi = d.shi[at + t], next_lo = d.slo[at + t], xv = Elem<T>::to_f32(x[t * x_token]);
        const float decay = __builtin_amdgcn_exp2f((next_hi - hi) + (next_lo - lo)), dx = d.dt[at + t] * xv;
        hi = next_hi;
        lo = next_lo;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < NP / 4; k += kVec<T>) {
            const int m = threadIdx.x % 4 * (NP / 4) + k;
            float bv[kVec<T>], cv[kVec<T>];
            widen<T>(load_vec<T>(B + t * b_token + m, d.N - m), bv);
            widen<T>(load_vec<T>(C + t * c_token + m, d.N - m), cv);
#pragma unroll
            for (int e = 0; e < kVec<T>; ++e) {
                v[k + e] = decay * v[k + e] + dx * bv[e];
                sum += v[k + e] * cv[e];
            }
        }
        sum += __shfl_xor(sum, 1, kWave);
        sum += __shfl_xor(sum, 2, kWave);
        T *to = y + (int64_t)t * d.H * d.P;
        if (mine && threadIdx.x % 4 == 0 && Elem<T>::to_f32(*to) * 0.f != 0.f) *to = Elem<T>::from_f32(sum + skip * xv);
    }
}

// y of a chunk for some heads of a group.  C . B is theirs together and stays in registers
// (transposed: rows i, columns t); each head scales it by its decays, which makes it the
// operand that x is multiplied by.  A wave has rows t of strips w and 7 - w (bfloat16), so
// that the four waves have the same share of the triangle i <= t and each operand from LDS
// serves two strips.  The scaled C . B enters the product as two bfloat16 terms (rounded to one it
// made the error of y up to 1.35 times its own rounding's; 6 us of 59), and so does the entering
// state (1.4 times where it dominates; 2 us), whose two parts with segments are joined in float32.
// y is rounded once, at the end.  A factor of zero in a matrix product does not keep what is not
// finite from the tokens before it, so a workgroup that made such a y goes over its own once more,
// token by token, and corrects those (the look at every y: 1 us of 59).  Bound by memory and vector
// instructions together: 2 x 8192 tokens bfloat16, 32 heads, P = N = 64: 59 us, 3.4 TB/s with the
// states; ragged prompts 4 x 4096, N = 128: 82 us; 65536 tokens float32, 2 heads, N = 64: 40 us, a
// little over half the rate of its matrix instructions.
template <typename T, int NP, bool WHOLE, bool SEG>
__global__ __launch_bounds__(kThreads, 2) void scan_out_kernel(OutArgs a, const T *__restrict__ X,
                                                               const T *__restrict__ Bm, const T *__restrict__ Cm,
                                                               T *__restrict__ y) {
    constexpr int QS = kStrips<T>, Q = 16 * QS, SPW = QS / 4;
    constexpr int LDN = ld_of<T>(NP), LDP = ld_of<T>(kSlab);
    constexpr bool TERMS = Elem<T>::is_bf16;  // the entering state's two
    constexpr int kTerm = kSlab * LDN, kTiles = Q * LDP + (TERMS ? 2 : 1) * kTerm;
    __shared__ __align__(16) T lds[kTiles > Q * LDN ? kTiles : Q * LDN];
    __shared__ __align__(16) float shi[Q], slo[Q], dts[Q];
    T *xtile = lds, *htile = lds + Q * LDP;
    const ScanDims &d = a.d;
    const int tid = threadIdx.x, lane = tid % kWave, wave = wave_of(tid), l16 = lane % 16, g = lane / 16;
    int id = (int)block_in_stretch();
    const int split = id % a.plan.splits;
    id /= a.plan.splits;
    const int grp = id % d.G;
    id /= d.G;
    const int c = id % d.nc, b = id / d.nc;
    const int rows = d.L - c * Q < Q ? d.L - c * Q : Q;  // rows of y
    int n = valid_tokens(d.lengths, b, d.L) - c * Q;
    n = n < 0 ? 0 : n > Q ? Q : n;
    const int hg = d.H / d.G, h0 = grp * hg + split * a.plan.per;
    const int h1 = h0 + a.plan.per < (grp + 1) * hg ? h0 + a.plan.per : (grp + 1) * hg;
    if (n == 0) {  // nothing of this chunk may be read
        const int64_t each = (int64_t)(h1 - h0) * d.P, tok = (int64_t)b * d.L + c * Q;
        for (int t = 0; t < rows; ++t)
            for (int64_t i = tid; i < each; i += kThreads) y[((tok + t) * d.H + h0) * d.P + i] = Elem<T>::from_f32(0.f);
        return;
    }
    const int slabs = (d.P + kSlab - 1) / kSlab, items = (h1 - h0) * slabs, cols = state_cols(d.N);
    const T *xb = X + b * a.x_batch + (int64_t)c * Q * a.x_token;
    const int first = SEG ? c / d.seg * d.seg : c;  // the chunk whose place has the entering state, or the segment's
    const bool has_h = n > 0 && (first > 0 || a.has_first), has_b = SEG && n > 0 && c > first;
    int strip[SPW];
    const int below = l16 - 4 * g;  // on the diagonal tile, row v of this lane is column t's token at v == below
#pragma unroll
    for (int j = 0; j < SPW; ++j) strip[j] = j == 0 ? wave : QS - 1 - wave;

    TileFetch<T, Q, kSlab, kThreads, WHOLE> xf;
    TileFetch<float, kSlab, NP, kThreads, true> hf;
    TileFetch<float, kSlab, NP, kThreads, true> bf;
    float tf[3], skip_next, carry_next = 1.f;
    auto fetch = [&](int it) {
        const int h = h0 + it / slabs, p0 = it % slabs * kSlab, tid = afresh(threadIdx.x);
        skip_next = a.D[h];
        xf.fetch(xb + (int64_t)h * d.P + p0, a.x_token, n, d.P - p0, tid);
        const int64_t chunk = ((int64_t)b * d.H + h) * d.nc + c;
        if (!SEG && has_h) hf.fetch(a.states + (chunk * d.P + p0) * cols, cols, d.P - p0, cols, tid);
        if (has_b) {
            carry_next = a.carried[chunk];
            bf.fetch(a.states + (chunk * d.P + p0) * cols, cols, d.P - p0, cols, tid);
        }
        if (tid < Q) {
            tf[0] = d.shi[chunk * Q + tid];
            tf[1] = d.slo[chunk * Q + tid];
            tf[2] = d.dt[chunk * Q + tid];
        }
    };

    // C of the wave's rows, and C . B for every i <= t
    Frag<T> cf[SPW][NP / 32];
    f32x4 cb[SPW][QS];
    {
        TileFetch<T, Q, NP, kThreads, false> cg, bg;
        cg.fetch(Cm + b * a.c_batch + (int64_t)c * Q * a.c_token + grp * d.N, a.c_token, n, d.N, tid);
        bg.fetch(Bm + b * a.b_batch + (int64_t)c * Q * a.b_token + grp * d.N, a.b_token, n, d.N, tid);
        cg.put(lds, LDN, n, d.N, tid);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < SPW; ++j)
#pragma unroll
            for (int k = 0; k < NP / 32; ++k) cf[j][k] = near_frag(lds + (16 * strip[j] + l16) * LDN + 32 * k, g);
        __syncthreads();
        bg.put(lds, LDN, n, d.N, tid);
        __syncthreads();
        fetch(0);
#pragma unroll
        for (int i = 0; i < QS; ++i) {
            Frag<T> bf[NP / 32];
#pragma unroll
            for (int k = 0; k < NP / 32; ++k) bf[k] = near_frag(lds + (16 * i + l16) * LDN + 32 * k, g);
#pragma unroll
            for (int j = 0; j < SPW; ++j) {
                cb[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (SPW == 2 && j == 0 && i >= QS / 2) continue;  // strip[0] is in the first half
#pragma unroll
                for (int k = 0; k < NP / 32; ++k) cb[j][i] = mma(bf[k], cf[j][k], cb[j][i]);
            }
        }
    }

    float largest = 0.f;  // of this lane's results; NaN counts as the largest
    for (int it = 0; it < items; ++it) {
        const int h = h0 + it / slabs, p0 = it % slabs * kSlab, tid = afresh(threadIdx.x);
        // not an item ahead like the rest: a segment's chunks read the same from the L2, and the registers of
        // both parts are too many (ragged prompts, N = 128: 27 spill, 167 -> 152 us; float32 pixels 75 -> 71)
        if (SEG && has_h) hf.fetch(a.states + ((((int64_t)b * d.H + h) * d.nc + first) * d.P + p0) * cols, cols, d.P - p0, cols, tid);
        __syncthreads();
        xf.put(xtile, LDP, n, d.P - p0, tid);
        const float carry = carry_next;
        if (has_h || has_b) {
#pragma unroll
            for (int k = 0; k < decltype(hf)::kCount; ++k) {
                f32x4 v = {0.f, 0.f, 0.f, 0.f};
                if (has_h) v = __builtin_bit_cast(f32x4, hf.r[k]);
                if constexpr (SEG)
                    if (has_b) v = v * carry + __builtin_bit_cast(f32x4, bf.r[k]);
                // zeros past the tensor, once for both parts
                if (hf.row_of(k, tid) >= d.P - p0 || hf.col_of(k, tid) >= cols) v = f32x4{0.f, 0.f, 0.f, 0.f};
                T *to = htile + hf.row_of(k, tid) * LDN + hf.col_of(k, tid);
                store4<T>(to, v, 4);
                if constexpr (TERMS) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] -= (float)(__bf16)v[e];
                    store4<T>(to + kTerm, v, 4);
                }
            }
        }
        if (tid < Q) {
            shi[tid] = tf[0];
            slo[tid] = tf[1];
            dts[tid] = tf[2];
        }
        __syncthreads();
        const float skip = skip_next;  // asked for with the item: a read here would wait for the next item's too
        if (it + 1 < items) fetch(it + 1);
        f32x4 acc[SPW][4];
#pragma unroll
        for (int j = 0; j < SPW; ++j)
#pragma unroll
            for (int p = 0; p < 4; ++p) acc[j][p] = f32x4{0.f, 0.f, 0.f, 0.f};
        float th[SPW], tl[SPW];
#pragma unroll
        for (int j = 0; j < SPW; ++j) {
            th[j] = shi[16 * strip[j] + l16];
            tl[j] = slo[16 * strip[j] + l16];
        }
        auto add_tile = [&](const T *tile) {
#pragma unroll
            for (int k = 0; k < NP / 32; ++k)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const Frag<T> hr = near_frag(tile + (16 * p + l16) * LDN + 32 * k, g);
#pragma unroll
                    for (int j = 0; j < SPW; ++j) acc[j][p] = mma(hr, cf[j][k], acc[j][p]);
                }
        };
        if (has_h || has_b) {
            add_tile(htile);
            if constexpr (TERMS) add_tile(htile + kTerm);
#pragma unroll
            for (int j = 0; j < SPW; ++j) {
                const float f = __builtin_amdgcn_exp2f(th[j] + tl[j]);
#pragma unroll
                for (int p = 0; p < 4; ++p) acc[j][p] *= f;
            }
        }
#pragma unroll
        for (int i = 0; i < QS / 2; ++i) {
            if (2 * i > strip[SPW - 1]) continue;
            Frag<T> xr[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) xr[p] = col_frag(xtile, LDP, 32 * i, 16 * p, l16, g);
#pragma unroll
            for (int j = 0; j < SPW; ++j) {
                if ((SPW == 2 && j == 0 && i >= QS / 4) || 2 * i > strip[j]) continue;
                f32x4 m[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int is = 2 * i + u;
                    m[u] = f32x4{0.f, 0.f, 0.f, 0.f};
                    if (is > strip[j]) continue;
                    const f32x4 ih = *(const f32x4 *)(shi + 16 * is + 4 * g), il = *(const f32x4 *)(slo + 16 * is + 4 * g);
                    const f32x4 id4 = *(const f32x4 *)(dts + 16 * is + 4 * g);
                    f32x4 dif;
#pragma unroll
                    for (int v = 0; v < 4; ++v) dif[v] = (th[j] - ih[v]) + (tl[j] - il[v]);
                    if (is == strip[j])
#pragma unroll
                        for (int v = 0; v < 4; ++v) dif[v] = v <= below ? dif[v] : -INFINITY;
#pragma unroll
                    for (int v = 0; v < 4; ++v) m[u][v] = cb[j][is][v] * (__builtin_amdgcn_exp2f(dif[v]) * id4[v]);
                }
                Frag<T> ml;
                const Frag<T> mf = pack_frag2<T>(m[0], m[1], ml);
#pragma unroll
                for (int p = 0; p < 4; ++p) acc[j][p] = mma2(xr[p], mf, ml, acc[j][p]);
            }
        }
#pragma unroll
        for (int j = 0; j < SPW; ++j) {
            const int t = 16 * strip[j] + l16;
            if (t >= rows) continue;
            T *yr = y + (((int64_t)b * d.L + c * Q + t) * d.H + h) * d.P + p0;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int at = 16 * p + 4 * g;
                f32x4 o = acc[j][p] + skip * lds4(xtile + t * LDP + at);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    o[v] = t < n ? o[v] : 0.f;
                    largest = __builtin_elementwise_maximum(largest, __builtin_fabsf(o[v]));
                }
                if (p0 + at < d.P) store4<T>(yr + at, o, WHOLE ? 4 : d.P - p0 - at);
            }
        }
    }
    if (!__syncthreads_or(!(largest < INFINITY))) return;
    for (int it = 0; it < items; ++it) {
        const int64_t head = (int64_t)b * d.H + h0 + it / slabs;
        const int p = it % slabs * kSlab + tid / 4;  // four threads a row of the state
        const bool mine = p < d.P;
        const float *place = a.states + (head * d.nc * d.P + (mine ? p : 0)) * cols;
        const float carry = has_b ? a.carried[head * d.nc + c] : 1.f;
        float v[NP / 4];
#pragma unroll
        for (int k = 0; k < NP / 4; ++k) {
            const int m = tid % 4 * (NP / 4) + k;
            v[k] = 0.f;
            if (m < cols) {
                if (has_h) v[k] = place[(int64_t)first * d.P * cols + m];
                if (has_b) v[k] = v[k] * carry + place[(int64_t)c * d.P * cols + m];
            }
        }
        // a row whose entering state is not finite has no y to correct
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < NP / 4; ++k) sum += v[k] * 0.f;
        sum += __shfl_xor(sum, 1, kWave);
        sum += __shfl_xor(sum, 2, kWave);
        T *yr = y + (((int64_t)b * d.L + c * Q) * d.H + h0 + it / slabs) * d.P + (mine ? p : 0);
        bool any = false;
        for (int t = tid % 4; mine && sum == 0.f && t < n; t += 4)
            any |= Elem<T>::to_f32(yr[(int64_t)t * d.H * d.P]) * 0.f != 0.f;
        if (!__any(any)) continue;
        recur<T, NP>(d, head, c, n, mine, v, xb + (int64_t)(h0 + it / slabs) * d.P + (mine ? p : 0), a.x_token,
                     Bm + b * a.b_batch + (int64_t)c * Q * a.b_token + grp * d.N, a.b_token,
                     Cm + b * a.c_batch + (int64_t)c * Q * a.c_token + grp * d.N, a.c_token, a.D[h0 + it / slabs], yr);
    }
}

// One token of each sequence.  The state's traffic is everything (8 bytes and 5 operations
// an element); LN lanes hold a row of N, V elements each, UNROLL rows a thread at once.  A
// slot outside [0, S) is a place without a sequence: y is zero and no state is touched.  256
// sequences, 32 heads, P = 64, N = 128: 92 us, 5.8 TB/s; one sequence of 2 heads, N = 64: 3.7 us.
template <typename T, int V, int UNROLL>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(Scan a, float *__restrict__ state,
                                                             const int *__restrict__ slots, int64_t S,
                                                             T *__restrict__ y, int ln, int blocks_p) {
    const int bp = blockIdx.x % blocks_p;
    const int64_t bh = blockIdx.x / blocks_p;
    const int h = (int)(bh % a.H);
    const int64_t b = bh / a.H;
    const int lane = threadIdx.x % ln, rows = kThreads / ln, r0 = bp * rows * UNROLL + threadIdx.x / ln;
    const int64_t slot = slots != nullptr ? slots[b] : b;
    const bool on = slot >= 0 && slot < S;
    const T *xr = (const T *)a.x + b * a.x_batch + (int64_t)h * a.P;
    T *yr = y + bh * a.P;
    if (!on) {
        for (int k = 0; k < UNROLL; ++k)
            if (lane == 0 && r0 + k * rows < a.P) yr[r0 + k * rows] = Elem<T>::from_f32(0.f);
        return;
    }
    const int grp = h / (a.H / a.G);
    const T *Bv = (const T *)a.Bm + b * a.b_batch + (int64_t)grp * a.N, *Cv = (const T *)a.Cm + b * a.c_batch + (int64_t)grp * a.N;
    float *st = state + (slot * a.H + h) * a.P * a.N;
    const float dt = softplus(Elem<T>::to_f32(((const T *)a.dt)[b * a.dt_batch + h]) + a.dt_bias[h]);
    const float decay = expf(dt * a.A[h]), skip = a.D[h];
    float sum[UNROLL], xv[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
        sum[k] = 0.f;
        xv[k] = r0 + k * rows < a.P ? Elem<T>::to_f32(xr[r0 + k * rows]) : 0.f;
    }
    for (int n = lane * V; n < a.N; n += ln * V) {  // one turn for N up to 64 V
        typedef float vec __attribute__((ext_vector_type(V), aligned(4)));
        vec v[UNROLL];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k)
            if (r0 + k * rows < a.P) v[k] = *(const vec *)(st + (int64_t)(r0 + k * rows) * a.N + n);
        float bv[V], cv[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            bv[e] = dt * Elem<T>::to_f32(Bv[n + e]);
            cv[e] = Elem<T>::to_f32(Cv[n + e]);
        }
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            if (r0 + k * rows >= a.P) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[k][e] = decay * v[k][e] + xv[k] * bv[e];
                sum[k] += v[k][e] * cv[e];
            }
            *(vec *)(st + (int64_t)(r0 + k * rows) * a.N + n) = v[k];
        }
    }
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
        for (int m = 1; m < ln; m *= 2) sum[k] += __shfl_xor(sum[k], m, kWave);
        if (lane == 0 && r0 + k * rows < a.P) yr[r0 + k * rows] = Elem<T>::from_f32(sum[k] + skip * xv[k]);
    }
}

namespace {

template <typename T>
hipError_t scan_fwd(const Scan &a, float *work, void *y, float *final_state, bool save, hipStream_t stream) {
    constexpr int Q = 16 * kStrips<T>;
    const ScanWork w = scan_work(a.B, a.L, a.H, a.P, a.G, a.N, Elem<T>::is_bf16, save);
    const ScanDims d = {(int)a.B, (int)a.L, a.H, a.P, a.G, a.N, w.nc, w.seg, a.lengths, work + w.dt, work + w.shi,
                        work + w.slo, work + w.decay};
    const int blocks_h = (a.H + kTimeHeads - 1) / kTimeHeads;
    const ChunkPlan plan = plan_heads(a.B, w.nc, a.H, a.P, a.G, 512);
    const int64_t bt = a.B * w.nc * blocks_h, bo = a.B * w.nc * a.G * plan.splits;
    if (bt > 0x7fffffff || bo > 0x7fffffff) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((scan_times_kernel<T>), dim3((unsigned)bt), dim3(kThreads), 0, stream, d, (const T *)a.dt, a.dt_batch,
                       a.dt_token, a.A, a.dt_bias, blocks_h);
    hipError_t e = hipGetLastError();
    float *states = work + w.states;
    if (e == hipSuccess && (w.nc > 1 || a.initial != nullptr || final_state != nullptr || save)) {
        if (w.seg > 1)
            e = launch_scan_segments<T>(d, w.hw, (const T *)a.x, a.x_batch, a.x_token, (const T *)a.Bm, a.b_batch,
                                        a.b_token, states, work + w.carried, work + w.decays, stream);
        else
            e = launch_scan_states<T>(d, (const T *)a.x, a.x_batch, a.x_token, (const T *)a.Bm, a.b_batch, a.b_token,
                                      states, false, stream);
        if (e == hipSuccess) e = launch_scan_pass(d, states, w.seg > 1 ? work + w.decays : d.decay, a.initial, final_state, Q, false, stream);
    }
    if (e != hipSuccess) return e;
    const OutArgs o = {d, plan, a.x_batch, a.x_token, a.b_batch, a.b_token, a.c_batch, a.c_token, states,
                       work + w.carried, a.initial != nullptr, a.D};
#define X_(NP, WHOLE)                                                                                              \
    if (w.seg > 1)                                                                                                 \
        hipLaunchKernelGGL((scan_out_kernel<T, NP, WHOLE, true>), dim3((unsigned)bo), dim3(kThreads), 0, stream,   \
                           o, (const T *)a.x, (const T *)a.Bm, (const T *)a.Cm, (T *)y);                           \
    else                                                                                                           \
        hipLaunchKernelGGL((scan_out_kernel<T, NP, WHOLE, false>), dim3((unsigned)bo), dim3(kThreads), 0, stream,  \
                           o, (const T *)a.x, (const T *)a.Bm, (const T *)a.Cm, (T *)y);
    DDPM_SEQ_SCAN_SHAPES(T, a.N, a.P, X_)
#undef X_
    return hipGetLastError();
}

template <typename T, int V>
hipError_t scan_step(const Scan &a, float *state, const int *slots, int64_t S, void *y, hipStream_t stream) {
    int ln = 1;
    while (ln < kWave && ln * V < a.N) ln *= 2;
    // rows at once: as many as still leave two workgroups a compute unit (8 and 1: 93 and 160 us for 256
    // sequences, 32 heads, 64 x 128; 6.3 and 4.8 us for one of 2 heads, 64 x 64)
    const int rows = kThreads / ln;
    int unroll = 8;
    while (unroll > 1 && (a.P <= rows * (unroll / 2) || a.B * a.H * ((a.P + rows * unroll - 1) / (rows * unroll)) < 512))
        unroll /= 2;
    const int blocks_p = (a.P + rows * unroll - 1) / (rows * unroll);
    const int64_t blocks = a.B * a.H * blocks_p;
    if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
#define X(U)                                                                                                           \
    if (unroll == U)                                                                                                   \
        hipLaunchKernelGGL((scan_step_kernel<T, V, U>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, a, state,   \
                           slots, S, (T *)y, ln, blocks_p);
    X(1) X(2) X(4) X(8)
#undef X
    return hipGetLastError();
}

template <typename T>
hipError_t scan_step(const Scan &a, float *state, const int *slots, int64_t S, void *y, hipStream_t stream) {
    if (a.N % 4 == 0) return scan_step<T, 4>(a, state, slots, S, y, stream);
    if (a.N % 2 == 0) return scan_step<T, 2>(a, state, slots, S, y, stream);
    return scan_step<T, 1>(a, state, slots, S, y, stream);
}

}  // namespace

int scan_chunk(bool bf16) { return 16 * (bf16 ? kStrips<bf16_t> : kStrips<float>); }

int64_t scan_fwd_floats(int64_t B, int64_t L, int H, int P, int G, int N, bool bf16) {
    const int64_t kept = scan_work(B, L, H, P, G, N, bf16, true).total, not_kept = scan_work(B, L, H, P, G, N, bf16, false).total;
    return kept > not_kept ? kept : not_kept;
}

hipError_t launch_scan_fwd(const Scan &a, float *work, void *y, float *final_state, bool save, bool bf16,
                           hipStream_t stream) {
    return bf16 ? scan_fwd<bf16_t>(a, work, y, final_state, save, stream)
                : scan_fwd<float>(a, work, y, final_state, save, stream);
}

hipError_t launch_scan_step(const Scan &a, float *state, const int *slots, int64_t S, void *y, bool bf16,
                            hipStream_t stream) {
    return bf16 ? scan_step<bf16_t>(a, state, slots, S, y, stream) : scan_step<float>(a, state, slots, S, y, stream);
}

}  // namespace seq
}  // namespace ddpm
