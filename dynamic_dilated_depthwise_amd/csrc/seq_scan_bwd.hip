// seq_scan_bwd.hip -- the selective scan's backward pass (seq_scan.hpp has the forward's
// formulas).
//
// For a chunk, with h0 the state that enters it, g1 the gradient that reaches its end from
// later tokens, E[t, i] = exp(s[t] - s[i]) for i <= t, CB[t, i] = C[t] . B[i] and
// Z[t, i] = grad[t] . x[i]:
//
//   grad_x[i] = dt[i] (sum_t CB E grad[t] + exp(s_end - s[i]) g1 B[i]) + D grad[i]
//   grad_B[i] = dt[i] (sum_t Z E C[t] + exp(s_end - s[i]) g1' x[i])      summed over heads
//   grad_C[t] = sum_i Z E dt[i] B[i] + exp(s[t]) h0' grad[t]             summed over heads
//
// The times.  Let r[t] = grad[t] . (y[t] - D x[t]) and q[i] = dt[i] * (what multiplies dt[i]
// x[i] in the sums above, dotted with x[i]).  The gradient of the decay that token t applies
// is what flows from tokens before t to t and later,
//
//   e[t] = exp(s_end) <g1, h0> + sum_{i < t} q_end[i] + sum_{k >= t} r_in[k]
//          + sum_{k >= t} (r_own[k] - q_own[k]),
//
// where q_end is q's part through g1, r_in r's part through h0, and r_own, q_own the parts
// inside the chunk.  What r_own and q_own share, the diagonal and the pairs after t,
// cancels: both add the very same float32 products, in 64 bits, so that no more than the
// other products' own roundings is left.  Then
// grad_dt = (q / dt + A e) sigmoid(raw + dt_bias) and grad_A = sum_t dt e.  These are sums
// of many terms of both signs, so every factor keeps float32's precision: Z and CB come
// from products of the inputs themselves, and h0 and g1 enter as three bfloat16 terms.
// grad_x, grad_B and grad_C take the scaled CB, Z and g1 in two terms (17 bits) and are rounded to
// bfloat16 at their end.
#include "seq_scan.hpp"

namespace ddpm {
namespace seq {

struct BwdArgs {
    ScanDims d;
    ChunkPlan plan;
    int64_t x_batch, x_token, b_batch, b_token, c_batch, c_token, g_batch, g_token;
    const float *states, *adjoints;  // [B, H, nc, P, cols]; adjoints null: nothing reaches the only chunk's end
    const float *A, *D;
    float *part;   // [splits, 2, B, L, G, N] or null (one split: grad_B and grad_C at once)
    double *heads;  // [3, H, B * nc]: every chunk's part of grad_A, grad_dt_bias, grad_D
    // for the sums over a head's tokens at a workgroup's end, [B, H, nc, Q]: r_in + r_own - q_own,
    // q_end, q / dt; and [B, H, nc, waves, 2]: the waves' parts of <g1, h0> and grad . x
    double *later, *qend, *direct, *marks;
    int has_first, has_last;  // an initial state, a gradient of the final one
};

template <typename T, int NP>
struct BwdLds {
    static constexpr int QS = kStrips<T>, Q = 16 * QS, LDN = ld_of<T>(NP);
    static constexpr int LDP = NP <= 64 ? ld_of<T>(kSlab) : kSlab + kVec<T>;  // 160 KB hold no more at 128
    T b[Q * LDN], c[Q * LDN], x[Q * LDP], g[Q * LDP];
    // h0 and g1: a set of planes each where 160 KB hold them, else g1 follows h0 into one
    static constexpr int kTilesBytes = 2 * Q * (LDN + LDP) * (int)sizeof(T) + 3 * Q * 4;
    static constexpr int kPlanes = kTerms<T> * kSlab * LDN;
    static constexpr int kSets = kTilesBytes + 2 * kPlanes * (int)sizeof(T) <= 160 * 1024 ? 2 : 1;
    T plane[kSets][kTerms<T>][kSlab * LDN];
    float shi[Q], slo[Q], dt[Q];
};

// Sum over the four lane groups that hold a column's rows.
template <typename V>
__device__ __forceinline__ V over_groups(V v) {
    v += __shfl_xor(v, 16, kWave);
    return v + __shfl_xor(v, 32, kWave);
}
template <typename V>
__device__ __forceinline__ V over_wave(V v) {
#pragma unroll
    for (int m = 1; m < kWave; m *= 2) v += __shfl_xor(v, m, kWave);
    return v;
}

__device__ __forceinline__ float frag_at(const bf16x8 &f, int e) { return (float)f[e]; }
__device__ __forceinline__ float frag_at(const FragF &f, int e) { return f.v[e]; }

// One chunk, some heads of a group.  A wave has a strip of the chunk's tokens both as rows t
// (grad_C, r) and as columns i (grad_x, grad_B, q).  Strips go in pairs, 32 of a contraction:
// a wave in pair kw has the pairs before kw as rows, those after it as columns, and its own as
// both, masked; the same work for every wave, and its tiles of C . B stay in registers.  Two waves
// a SIMD with all registers taken; a head costs a wave 1660 vector, 144 matrix and 285 LDS
// instructions, and those three and the barriers around the tiles add up more than they overlap
// (vector issue 50 %, LDS 30 %, matrix 17 % of the time): 2 x 8192 tokens bfloat16, 32 heads, P =
// N = 64: 200 us.  N = 128 takes 580 us: one set of planes, and 130 registers spill.
template <typename T, int NP, bool WHOLE>
__global__ __launch_bounds__(64 * kStrips<T>) void scan_bwd_kernel(BwdArgs a, const T *__restrict__ X,
                                                                   const T *__restrict__ Bm, const T *__restrict__ Cm,
                                                                   const T *__restrict__ grad, T *__restrict__ grad_x,
                                                                   T *__restrict__ grad_dt, T *__restrict__ grad_B,
                                                                   T *__restrict__ grad_C) {
    typedef BwdLds<T, NP> Lds;
    constexpr int WAVES = Lds::QS, Q = Lds::Q, THREADS = 64 * WAVES, SETS = Lds::kSets;
    constexpr int LDN = Lds::LDN, LDP = Lds::LDP, NS = NP / 16;
    extern __shared__ __align__(16) char raw_lds[];
    Lds &s = *(Lds *)raw_lds;
    const ScanDims &d = a.d;
    const int tid = threadIdx.x, lane = tid % kWave, wave = wave_of(tid), l16 = lane % 16, g = lane / 16;
    int id = (int)block_in_stretch();
    const int split = id % a.plan.splits;
    id /= a.plan.splits;
    const int grp = id % d.G;
    id /= d.G;
    const int c = id % d.nc, b = id / d.nc;
    const int rows = d.L - c * Q < Q ? d.L - c * Q : Q;
    const int len = valid_tokens(d.lengths, b, d.L);
    int n = len - c * Q;
    n = n < 0 ? 0 : n > Q ? Q : n;
    const int hg = d.H / d.G, h0 = grp * hg + split * a.plan.per;
    const int h1 = h0 + a.plan.per < (grp + 1) * hg ? h0 + a.plan.per : (grp + 1) * hg;
    const int slabs = (d.P + kSlab - 1) / kSlab, items = (h1 - h0) * slabs, cols = state_cols(d.N);
    const int64_t tok0 = (int64_t)b * d.L + c * Q;  // first token's row in the contiguous outputs
    const bool has_h = n > 0 && (c > 0 || a.has_first), has_g = (c + 1) * Q < len || (a.has_last && n > 0);
    const T *xb = X + b * a.x_batch + (int64_t)c * Q * a.x_token;
    const T *gb = grad + b * a.g_batch + (int64_t)c * Q * a.g_token;
    const int kw = wave / 2;
    const int me = 16 * wave + l16;  // this lane's token, as row t and as column i

    TileFetch<T, Q, kSlab, THREADS, WHOLE> xf, gf;
    TileFetch<float, kSlab, NP, THREADS, true> hf, af;
    float tf[3], skip_next;
    auto chunk_of = [&](int it) { return ((int64_t)b * d.H + h0 + it / slabs) * d.nc + c; };
    auto fetch_adjoint = [&](int it) {
        const int p0 = it % slabs * kSlab, tid = afresh(threadIdx.x);
        if (has_g) af.fetch(a.adjoints + (chunk_of(it) * d.P + p0) * cols, cols, d.P - p0, cols, tid);
    };
    // an item's operands; with one set of planes the adjoint is asked for when the one before has been used
    auto fetch = [&](int it) {
        const int h = h0 + it / slabs, p0 = it % slabs * kSlab, tid = afresh(threadIdx.x);
        const int64_t chunk = chunk_of(it);
        skip_next = a.D[h];
        if (tid < Q) {
            tf[0] = d.shi[chunk * Q + tid];
            tf[1] = d.slo[chunk * Q + tid];
            tf[2] = d.dt[chunk * Q + tid];
        }
        if (!WHOLE || n > 0) {  // nothing of a chunk past the length may be read (vectors of parts are not)
            xf.fetch(xb + (int64_t)h * d.P + p0, a.x_token, n, d.P - p0, tid);
            gf.fetch(gb + (int64_t)h * d.P + p0, a.g_token, n, d.P - p0, tid);
        }
        if (has_h) hf.fetch(a.states + (chunk * d.P + p0) * cols, cols, d.P - p0, cols, tid);
        if (SETS == 2) fetch_adjoint(it);
    };
    // A float32 tile into a set of planes.  `dot` gains the adjoint's product with the state: with
    // one set the state is what this thread put there before.
    float dot = 0.f;
    auto put_planes = [&](const decltype(hf) &f, int set, int p0, bool against) {
        const int tid = afresh(threadIdx.x);
#pragma unroll
        for (int k = 0; k < decltype(hf)::kCount; ++k) {
            if (!hf.has(k, tid)) continue;
            const int at = f.row_of(k, tid) * LDN + f.col_of(k, tid);
            float v[4];
            widen<float>(f.get(k, d.P - p0, cols, tid), v);
            if (against && SETS == 2) {
                float w[4];
                widen<float>(hf.get(k, d.P - p0, cols, tid), w);
#pragma unroll
                for (int e = 0; e < 4; ++e) dot += v[e] * w[e];
            }
            if constexpr (Elem<T>::is_bf16) {
                if (against && SETS == 1) {
                    u16x4 t[3];
#pragma unroll
                    for (int m = 0; m < 3; ++m) t[m] = *(const u16x4 *)(s.plane[0][m] + at);
#pragma unroll
                    for (int e = 0; e < 4; ++e)  // the three terms' sum is the float32 that they came from
                        dot += v[e] * (bf16_bits_to_f32(t[0][e]) + (bf16_bits_to_f32(t[1][e]) + bf16_bits_to_f32(t[2][e])));
                }
                u16x4 t[3];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    __bf16 q0, q1, q2;
                    split3(v[e], q0, q1, q2);
                    t[0][e] = __builtin_bit_cast(uint16_t, q0);
                    t[1][e] = __builtin_bit_cast(uint16_t, q1);
                    t[2][e] = __builtin_bit_cast(uint16_t, q2);
                }
#pragma unroll
                for (int m = 0; m < 3; ++m) *(u16x4 *)(s.plane[set][m] + at) = t[m];
            } else {
                if (against && SETS == 1) {
                    const f32x4 t = *(const f32x4 *)(s.plane[0][0] + at);
#pragma unroll
                    for (int e = 0; e < 4; ++e) dot += v[e] * t[e];
                }
                *(f32x4 *)(s.plane[set][0] + at) = f32x4{v[0], v[1], v[2], v[3]};
            }
        }
    };
    // The sums over the tokens of a head: one wave, Q / 64 tokens a lane.
    auto finish_head = [&](int h) {
        constexpr int PER = Q / kWave;
        const int64_t chunk = ((int64_t)b * d.H + h) * d.nc + c, at = chunk * Q + lane * PER;
        double dot = 0., diag = 0.;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            dot += a.marks[(chunk * WAVES + w) * 2];
            diag += a.marks[(chunk * WAVES + w) * 2 + 1];
        }
        double pre[PER], suf[PER], before = 0., after = 0.;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            pre[e] = before;
            before += a.qend[at + e];
        }
#pragma unroll
        for (int e = PER - 1; e >= 0; --e) {
            after += a.later[at + e];
            suf[e] = after;
        }
        double up = before, down = after;
#pragma unroll
        for (int m = 1; m < kWave; m *= 2) {
            const double u = __shfl_up(up, m, kWave), o = __shfl_down(down, m, kWave);
            if (lane >= m) up += u;
            if (lane + m < kWave) down += o;
        }
        up -= before;
        down -= after;
        const double A = a.A[h], end = d.decay[chunk];
        double sum_a = 0., sum_b = 0.;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int t = lane * PER + e;
            const float dt = d.dt[at + e];
            const double flow = end * dot + (up + pre[e]) + (down + suf[e]);
            // softplus's derivative from its value: 1 - exp(-dt)
            const double raw = t < n ? (a.direct[at + e] + A * flow) * -expm1f(-dt) : 0.;
            sum_a += t < n ? dt * flow : 0.;
            sum_b += raw;
            if (t < rows) grad_dt[(tok0 + t) * d.H + h] = Elem<T>::from_f32((float)raw);
        }
        sum_a = over_wave(sum_a);
        sum_b = over_wave(sum_b);
        if (lane == 0) {
            const int64_t M = (int64_t)d.B * d.nc, to = (int64_t)h * M + (int64_t)b * d.nc + c;
            a.heads[to] = sum_a;
            a.heads[d.H * M + to] = sum_b;
            a.heads[2 * d.H * M + to] = diag;
        }
    };

    // B and C, and the tiles of C . B: as rows transposed, D[i][t], as columns D[t][i].  Slot k
    // is pair k as rows for k < kw and pair k + 1 as columns from kw on.
    constexpr int SLOTS = WAVES / 2 - 1;
    f32x4 cbs[SLOTS][2], cbr[2], cbc[2];
    {
        TileFetch<T, Q, NP, THREADS, false> bf, cf;
        bf.fetch(Bm + b * a.b_batch + (int64_t)c * Q * a.b_token + grp * d.N, a.b_token, n, d.N, tid);
        cf.fetch(Cm + b * a.c_batch + (int64_t)c * Q * a.c_token + grp * d.N, a.c_token, n, d.N, tid);
        bf.put(s.b, LDN, n, d.N, tid);
        cf.put(s.c, LDN, n, d.N, tid);
        fetch(0);
        if (SETS == 1) fetch_adjoint(0);
        __syncthreads();
        auto tiles = [&](const T *rows_of, int strip, const T *cols_of, f32x4 (&r)[2], int u) {
            r[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < NP / 32; ++k) {
                const Frag<T> f = near_frag(rows_of + (16 * strip + l16) * LDN + 32 * k, g);
                r[u] = mma(f, near_frag(cols_of + me * LDN + 32 * k, g), r[u]);
            }
        };
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int k = 0; k < SLOTS; ++k) {
                if (k < kw) tiles(s.b, 2 * k + u, s.c, cbs[k], u);
                else tiles(s.c, 2 * k + 2 + u, s.b, cbs[k], u);
            }
            tiles(s.b, 2 * kw + u, s.c, cbr, u);
            tiles(s.c, 2 * kw + u, s.b, cbc, u);
        }
    }
    f32x4 dB[NS], dC[NS];
#pragma unroll
    for (int k = 0; k < NS; ++k) dB[k] = dC[k] = f32x4{0.f, 0.f, 0.f, 0.f};

    double rown = 0., qown = 0.;
    float rin = 0.f, qdt = 0.f, qend = 0.f, zdiag = 0.f;
    for (int it = 0; it < items; ++it) {
        const int h = h0 + it / slabs, slab = it % slabs, p0 = slab * kSlab;
        const int64_t chunk = chunk_of(it);
        const int tid = afresh(threadIdx.x);
        __syncthreads();
        xf.put(s.x, LDP, n, d.P - p0, tid);
        gf.put(s.g, LDP, n, d.P - p0, tid);
        if (has_h) put_planes(hf, 0, p0, false);
        if (SETS == 2 && has_g) put_planes(af, SETS - 1, p0, has_h);
        if (tid < Q) {
            s.shi[tid] = tf[0];
            s.slo[tid] = tf[1];
            s.dt[tid] = tf[2];
        }
        __syncthreads();
        const float skip = skip_next;  // asked for with the item: a read here would wait for the next item's too
        if (it + 1 < items) fetch(it + 1);
        const float mhi = s.shi[me], mlo = s.slo[me], mdt = s.dt[me];
        Frag<T> xr[2], gr[2];
        f32x4 dx[4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            xr[q] = near_frag(s.x + me * LDP + 32 * q, g);
            gr[q] = near_frag(s.g + me * LDP + 32 * q, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) zdiag += frag_at(xr[q], e) * frag_at(gr[q], e);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) dx[p] = f32x4{0.f, 0.f, 0.f, 0.f};
        // in the own pair, row 16 u + 4 g + v is this lane's token at 16 u + v == below
        const int below = afresh(me) - 32 * kw - 4 * g;
        // a pair of strips i = 2 k, 2 k + 1 against the wave's rows t
        auto as_rows = [&](int k, const f32x4 (&cb)[2], bool own) {
            f32x4 wt[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int is = 2 * k + u;
                const Frag<T> x0 = near_frag(s.x + (16 * is + l16) * LDP, g), x1 = near_frag(s.x + (16 * is + l16) * LDP + 32, g);
                const f32x4 ih = *(const f32x4 *)(s.shi + 16 * is + 4 * g), il = *(const f32x4 *)(s.slo + 16 * is + 4 * g);
                const f32x4 id4 = *(const f32x4 *)(s.dt + 16 * is + 4 * g);
                f32x4 z = {0.f, 0.f, 0.f, 0.f}, dif;
                z = mma(x1, gr[1], mma(x0, gr[0], z));
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    dif[v] = (mhi - ih[v]) + (mlo - il[v]);
                    if (own) dif[v] = 16 * u + v <= below ? dif[v] : -INFINITY;
                    wt[u][v] = z[v] * (__builtin_amdgcn_exp2f(dif[v]) * id4[v]);
                    rown += cb[u][v] * wt[u][v];  // the columns add the very same products
                }
            }
            Frag<T> wl;
            const Frag<T> wf = pack_frag2<T>(wt[0], wt[1], wl);
#pragma unroll
            for (int m = 0; m < NS; ++m) {
                const Frag<T> f = col_frag(s.b, LDN, 32 * k, 16 * m, l16, g);
                dC[m] = mma2(f, wf, wl, dC[m]);
            }
        };
        // a pair of strips t = 2 k, 2 k + 1 against the wave's columns i
        auto as_columns = [&](int k, const f32x4 (&cb)[2], bool own) {
            f32x4 nt[2], wt[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int ts = 2 * k + u;
                const Frag<T> g0 = near_frag(s.g + (16 * ts + l16) * LDP, g), g1 = near_frag(s.g + (16 * ts + l16) * LDP + 32, g);
                const f32x4 th = *(const f32x4 *)(s.shi + 16 * ts + 4 * g), tl = *(const f32x4 *)(s.slo + 16 * ts + 4 * g);
                f32x4 z = {0.f, 0.f, 0.f, 0.f}, dif;
                z = mma(g1, xr[1], mma(g0, xr[0], z));
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    dif[v] = (th[v] - mhi) + (tl[v] - mlo);
                    if (own) dif[v] = 16 * u + v >= below ? dif[v] : -INFINITY;
                    const float e = __builtin_amdgcn_exp2f(dif[v]);
                    nt[u][v] = cb[u][v] * e;
                    wt[u][v] = z[v] * (e * mdt);
                    qown += cb[u][v] * wt[u][v];
                    qdt += nt[u][v] * z[v];
                }
            }
            Frag<T> nl, wl;
            const Frag<T> nf = pack_frag2<T>(nt[0], nt[1], nl);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const Frag<T> f = col_frag(s.g, LDP, 32 * k, 16 * p, l16, g);
                dx[p] = mma2(f, nf, nl, dx[p]);
            }
            const Frag<T> wf = pack_frag2<T>(wt[0], wt[1], wl);
#pragma unroll
            for (int m = 0; m < NS; ++m) {
                const Frag<T> f = col_frag(s.c, LDN, 32 * k, 16 * m, l16, g);
                dB[m] = mma2(f, wf, wl, dB[m]);
            }
        };
        as_rows(kw, cbr, true);
        as_columns(kw, cbc, true);
#pragma unroll
        for (int k = 0; k < SLOTS; ++k) {
            if (k < kw) as_rows(k, cbs[k], false);
            else as_columns(k + 1, cbs[k], false);
        }
        if (has_h) {
            f32x4 o[NS];
#pragma unroll
            for (int m = 0; m < NS; ++m) o[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const Frag<T> go = row_frag(s.g + me * LDP + 32 * q, g);
#pragma unroll
                for (int t = 0; t < kTerms<T>; ++t)
#pragma unroll
                    for (int m = 0; m < NS; ++m) {
                        const Frag<T> f = col_frag(s.plane[0][t], LDN, 32 * q, 16 * m, l16, g);
                        o[m] = mma(f, go, o[m]);
                    }
            }
            const float f = __builtin_amdgcn_exp2f(mhi + mlo);
#pragma unroll
            for (int m = 0; m < NS; ++m) {
                o[m] *= f;
                dC[m] += o[m];
                const f32x4 cv = lds4(s.c + me * LDN + 16 * m + 4 * g);
#pragma unroll
                for (int v = 0; v < 4; ++v) rin += o[m][v] * cv[v];
            }
        }

        if (SETS == 1 && has_g) {
            __syncthreads();
            put_planes(af, 0, p0, has_h);
            if (it + 1 < items) fetch_adjoint(it + 1);
            __syncthreads();
        }
        if (has_g) {
            f32x4 o[4], w[NS];
#pragma unroll
            for (int p = 0; p < 4; ++p) o[p] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < NS; ++m) w[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < NP / 32; ++k) {
                const Frag<T> br = near_frag(s.b + me * LDN + 32 * k, g);
#pragma unroll
                for (int t = 0; t < kTerms<T>; ++t)
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const Frag<T> f = near_frag(s.plane[SETS - 1][t] + (16 * p + l16) * LDN + 32 * k, g);
                        o[p] = mma(f, br, o[p]);
                    }
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const Frag<T> xo = row_frag(s.x + me * LDP + 32 * q, g);
#pragma unroll
                for (int t = 0; t < (kTerms<T> > 1 ? 2 : 1); ++t)
#pragma unroll
                    for (int m = 0; m < NS; ++m) {
                        const Frag<T> f = col_frag(s.plane[SETS - 1][t], LDN, 32 * q, 16 * m, l16, g);
                        w[m] = mma(f, xo, w[m]);
                    }
            }
            const float f1 = __builtin_amdgcn_exp2f((s.shi[Q - 1] - mhi) + (s.slo[Q - 1] - mlo)), f2 = f1 * mdt;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                o[p] *= f1;
                dx[p] += o[p];
                const f32x4 xv = lds4(s.x + me * LDP + 16 * p + 4 * g);
#pragma unroll
                for (int v = 0; v < 4; ++v) qend += o[p][v] * xv[v];
            }
#pragma unroll
            for (int m = 0; m < NS; ++m) dB[m] += w[m] * f2;
        }
        if (me < rows) {
            T *o = grad_x + ((tok0 + me) * d.H + h) * d.P + p0;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int at = 16 * p + 4 * g;
                f32x4 r = dx[p] * mdt + skip * lds4(s.g + me * LDP + at);
#pragma unroll
                for (int v = 0; v < 4; ++v) r[v] = me < n ? r[v] : 0.f;
                if (p0 + at < d.P) store4<T>(o + at, r, WHOLE ? 4 : d.P - p0 - at);
            }
        }
        if (slab + 1 == slabs) {
            const double later = over_groups(rin + (rown - qown)), q0 = over_groups((double)qdt), q1 = over_groups((double)qend);
            if (g == 0) {
                const int64_t at = chunk * Q + me;
                a.later[at] = later;
                a.direct[at] = q0 + q1;
                a.qend[at] = mdt * q1;
            }
            rown = qown = 0.;
            rin = qdt = qend = 0.f;
            const double all_dot = over_wave((double)dot), diag = over_wave((double)zdiag);
            if (lane == 0) {
                a.marks[(chunk * WAVES + wave) * 2] = all_dot;
                a.marks[(chunk * WAVES + wave) * 2 + 1] = diag;
            }
            dot = zdiag = 0.f;
        }
    }
    __syncthreads();
    for (int h = h0 + wave; h < h1; h += WAVES) finish_head(h);

    if (me >= rows) return;
    const int64_t at = ((tok0 + me) * d.G + grp) * d.N;
    const int64_t all = (int64_t)d.B * d.L * d.G * d.N;
#pragma unroll
    for (int m = 0; m < NS; ++m) {
        const int k = 16 * m + 4 * g;
        if (k >= d.N) continue;
        if (a.part != nullptr) {
            store4<float>(a.part + 2 * split * all + at + k, dB[m], d.N - k);
            store4<float>(a.part + (2 * split + 1) * all + at + k, dC[m], d.N - k);
        } else {
            store4<T>(grad_B + at + k, dB[m], d.N - k);
            store4<T>(grad_C + at + k, dC[m], d.N - k);
        }
    }
}

// grad_B and grad_C from the splits' parts (in their order), and the heads' sums over all
// chunks (a wave a sum, in 64 bits).
template <typename T>
__global__ __launch_bounds__(256) void scan_bwd_sum_kernel(const float *__restrict__ part, int splits, int64_t all,
                                                           T *__restrict__ grad_B, T *__restrict__ grad_C,
                                                           const double *__restrict__ heads, int H, int64_t chunks,
                                                           float *__restrict__ grad_A, float *__restrict__ grad_bias,
                                                           float *__restrict__ grad_D, int64_t blocks_part) {
    if (blockIdx.x < blocks_part) {
        const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
        if (i >= 2 * all) return;
        const int left = 2 * all - i < 4 ? (int)(2 * all - i) : 4;
        f32x4 t = load4(part + i, left);
        for (int s = 1; s < splits; ++s) t += load4(part + 2 * s * all + i, left);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) (i + e < all ? grad_B + i + e : grad_C + i + e - all)[0] = Elem<T>::from_f32(t[e]);
        return;
    }
    const int64_t k = (blockIdx.x - blocks_part) * 4 + threadIdx.x / kWave;
    if (k >= 3 * H) return;
    double t = 0.;
    for (int64_t c = threadIdx.x % kWave; c < chunks; c += kWave) t += heads[k * chunks + c];
#pragma unroll
    for (int m = 1; m < kWave; m *= 2) t += __shfl_xor(t, m, kWave);
    if (threadIdx.x % kWave == 0) (k < H ? grad_A + k : k < 2 * H ? grad_bias + k - H : grad_D + k - 2 * H)[0] = (float)t;
}

namespace {

struct BwdWork {
    ChunkPlan plan;
    int64_t adjoints, heads, later, qend, direct, marks, part, total;
};
BwdWork bwd_work(int64_t B, int64_t L, int H, int P, int G, int N, int Q) {
    const int64_t nc = (L + Q - 1) / Q;
    BwdWork w;
    w.plan = plan_heads(B, nc, H, P, G, 256);
    w.adjoints = 0;
    w.heads = pad64(B * H * nc * P * state_cols(N));
    const int64_t tokens = pad64(2 * B * H * nc * Q);  // these and what follows to `part` in 64 bits
    w.later = w.heads + pad64(6 * H * B * nc);
    w.qend = w.later + tokens;
    w.direct = w.qend + tokens;
    w.marks = w.direct + tokens;
    w.part = w.marks + pad64(4 * B * H * nc * (Q / 16));
    w.total = w.part + (w.plan.splits > 1 ? pad64(2 * w.plan.splits * B * L * G * N) : 0);
    return w;
}

template <typename T, int NP, bool WHOLE>
hipError_t launch_main(const BwdArgs &k, int64_t blocks, const Scan &a, const void *grad, void *grad_x, void *grad_dt,
                       void *grad_B, void *grad_C, hipStream_t stream) {
    constexpr int bytes = sizeof(BwdLds<T, NP>);
    static_assert(bytes <= 160 * 1024, "a workgroup's LDS");
    auto kern = scan_bwd_kernel<T, NP, WHOLE>;
    hipError_t e = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(64 * kStrips<T>), bytes, stream, k, (const T *)a.x,
                       (const T *)a.Bm, (const T *)a.Cm, (const T *)grad, (T *)grad_x, (T *)grad_dt, (T *)grad_B,
                       (T *)grad_C);
    return hipGetLastError();
}

template <typename T>
hipError_t scan_bwd(const Scan &a, const float *saved, const void *grad, int64_t g_batch, int64_t g_token,
                    const float *grad_state, float *work, void *grad_x, void *grad_dt, float *grad_A, void *grad_B,
                    void *grad_C, float *grad_D, float *grad_dt_bias, float *grad_initial, hipStream_t stream) {
    constexpr int Q = 16 * kStrips<T>;
    const ScanWork f = scan_work(a.B, a.L, a.H, a.P, a.G, a.N, Elem<T>::is_bf16, true);
    const BwdWork w = bwd_work(a.B, a.L, a.H, a.P, a.G, a.N, Q);
    float *sv = const_cast<float *>(saved);  // only read here
    const ScanDims d = {(int)a.B, (int)a.L, a.H, a.P, a.G, a.N, f.nc, 1, a.lengths, sv + f.dt, sv + f.shi, sv + f.slo,
                        sv + f.decay};
    const int64_t blocks = a.B * f.nc * a.G * w.plan.splits, all = a.B * a.L * a.G * a.N;
    const int64_t blocks_part = w.plan.splits > 1 ? (2 * all + 1023) / 1024 : 0, blocks_sum = blocks_part + (3 * a.H + 3) / 4;
    if (blocks > 0x7fffffff || blocks_sum > 0x7fffffff) return hipErrorInvalidConfiguration;
    float *adjoints = nullptr;
    hipError_t e = hipSuccess;
    if (f.nc > 1 || grad_state != nullptr || grad_initial != nullptr) {
        adjoints = work + w.adjoints;
        e = launch_scan_states<T>(d, (const T *)grad, g_batch, g_token, (const T *)a.Cm, a.c_batch, a.c_token, adjoints,
                                  true, stream);
        if (e == hipSuccess) e = launch_scan_pass(d, adjoints, d.decay, grad_state, grad_initial, Q, true, stream);
    }
    if (e != hipSuccess) return e;
    const BwdArgs k = {d, w.plan, a.x_batch, a.x_token, a.b_batch, a.b_token, a.c_batch, a.c_token, g_batch, g_token,
                       saved + f.states, adjoints, a.A, a.D, w.plan.splits > 1 ? work + w.part : nullptr,
                       (double *)(work + w.heads), (double *)(work + w.later), (double *)(work + w.qend),
                       (double *)(work + w.direct), (double *)(work + w.marks),
                       a.initial != nullptr, grad_state != nullptr};
#define X_(NP, WHOLE) e = launch_main<T, NP, WHOLE>(k, blocks, a, grad, grad_x, grad_dt, grad_B, grad_C, stream);
    DDPM_SEQ_SCAN_SHAPES(T, a.N, a.P, X_)
#undef X_
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((scan_bwd_sum_kernel<T>), dim3((unsigned)blocks_sum), dim3(256), 0, stream, k.part,
                       w.plan.splits, all, (T *)grad_B, (T *)grad_C, k.heads, a.H, a.B * f.nc, grad_A, grad_dt_bias,
                       grad_D, blocks_part);
    return hipGetLastError();
}

}  // namespace

int64_t scan_bwd_floats(int64_t B, int64_t L, int H, int P, int G, int N, bool bf16) {
    return bwd_work(B, L, H, P, G, N, scan_chunk(bf16)).total;
}

hipError_t launch_scan_bwd(const Scan &a, const float *saved, const void *grad, int64_t g_batch, int64_t g_token,
                           const float *grad_state, float *work, void *grad_x, void *grad_dt, float *grad_A,
                           void *grad_B, void *grad_C, float *grad_D, float *grad_dt_bias, float *grad_initial,
                           bool bf16, hipStream_t stream) {
    return bf16 ? scan_bwd<bf16_t>(a, saved, grad, g_batch, g_token, grad_state, work, grad_x, grad_dt, grad_A, grad_B,
                                   grad_C, grad_D, grad_dt_bias, grad_initial, stream)
                : scan_bwd<float>(a, saved, grad, g_batch, g_token, grad_state, work, grad_x, grad_dt, grad_A, grad_B,
                                  grad_C, grad_D, grad_dt_bias, grad_initial, stream);
}

}  // namespace seq
}  // namespace ddpm
