// seq_scan.hpp -- what the selective scan's kernels share.
//
//   dt[t] = softplus(raw[t] + dt_bias),  a[t] = exp(dt[t] * A)           (per head)
//   h[t] = a[t] * h[t - 1] + dt[t] * x[t] (outer) B[t],   y[t] = h[t] C[t] + D * x[t]
//
// The sequence is cut into chunks of Q tokens.  With s[t] the running sum of dt * A from
// the chunk's first token on (inclusive) and h0 the state that enters the chunk,
//
//   y[t] = exp(s[t]) h0 C[t] + sum_{i <= t} (C[t] . B[i]) exp(s[t] - s[i]) dt[i] x[i] + D x[t]
//   h1   = exp(s[Q-1]) h0 + sum_i exp(s[Q-1] - s[i]) dt[i] x[i] (outer) B[i]
//
// so everything but the short recurrence over the chunks is a matrix product.  The kernels:
//   times    dt and s of every token (s in units of log2)
//   states   each chunk's own part of h1, all chunks at once
//   pass     the recurrence over the chunks, in place: the part becomes the h0 of its chunk
//   outputs  y of every chunk
// A call that keeps nothing for a backward moves fewer states: `segments` in the place of
// `states` runs the recurrence itself over a few chunks and writes what enters each of them
// from the segment's own tokens, in float32 as all states; `pass` then goes over segments only, and
// `outputs` adds the two parts of h0.
// The backward runs the same states and pass kernels over the chunks in reverse for the
// gradient that enters each chunk's end (with grad and C in the place of x and B) and one
// kernel for everything else.
//
// s is a difference of long sums, and its error is the relative error of a decay: it is
// summed in 64 bits and kept as two float32, hi + lo; hi's differences are exact where
// they are small, which is where the decay is not.
#pragma once

#include "seq_common.hpp"
#include "seq_launch.hpp"

namespace ddpm {
namespace seq {

constexpr int kSlab = 64;  // rows of the state (of P) that a workgroup works on at a time

// Tokens of a chunk, in strips of 16.  bfloat16: 128, so that the states in memory, which
// shrink with the chunk, and the products inside a chunk, which grow with it, cost about
// the same (training at 2 x 8192 tokens, 32 heads, P = N = 64: 372 us, with 64 tokens 515 us;
// ragged prompts 4 x 4096, 32 heads, N = 128: 152 and 213 us).  float32: 64, since its matrix
// products cost 16 times as much.
template <typename T> constexpr int kStrips = Elem<T>::is_bf16 ? 8 : 4;

struct ScanDims {
    int B, L, H, P, G, N, nc, seg;  // nc: chunks; seg: chunks of a segment (1: every chunk has its state)
    const int *lengths;
    float *dt, *shi, *slo;  // [B, H, nc * Q]
    float *decay;           // [B, H, nc]: exp of each chunk's whole sum
};

// Rows of N of the states in the workspaces start at multiples of four: [P, state_cols(N)],
// zeros behind N.
__host__ __device__ constexpr int state_cols(int N) { return (N + 3) / 4 * 4; }

struct ChunkPlan {
    int per, splits;  // heads of a workgroup; workgroups that share a chunk and a group
};

// Workgroups over (batch, chunk, group, split of the group's heads).  Heads of one group
// share B and C, which a workgroup prepares first, at about the cost of a head: the split with
// the shortest time for `slots` workgroups at once, in rounds of (heads + 1), and the fewest
// workgroups among equals.  (Training in bfloat16 at 2 x 64 chunks, 32 heads, with 2 and with 4
// splits in the backward: 356 and 366 us.)
inline ChunkPlan plan_heads(int64_t B, int64_t nc, int H, int P, int G, int64_t slots) {
    const int64_t base = B * nc * G, slabs = (P + kSlab - 1) / kSlab;
    const int hg = H / G;
    ChunkPlan best = {hg, 1};
    int64_t least = -1;
    for (int splits = 1; splits <= hg; ++splits) {
        const int per = (hg + splits - 1) / splits;
        const int64_t rounds = (base * ((hg + per - 1) / per) + slots - 1) / slots, cost = rounds * (per * slabs + 1);
        if (least < 0 || cost < least) {
            least = cost;
            best = {per, (hg + per - 1) / per};
        }
    }
    return best;
}

__device__ __forceinline__ int valid_tokens(const int *lengths, int b, int L) {
    if (lengths == nullptr) return L;
    const int n = lengths[b];
    return n < 0 ? 0 : n > L ? L : n;
}

inline int64_t pad64(int64_t n) { return (n + 63) / 64 * 64; }

// Segments of a call that keeps nothing: the longest, up to 8 chunks, and the most heads at
// once, up to 2, that leave 512 workgroups.  seg = 1: none, every chunk has its state.  With
// segments and without: ragged prompts 4 x 4096 bfloat16, 32 heads, P = 64, N = 128: 152 and 172 us;
// 65536 tokens float32, 2 heads, P = N = 64: 71 and 80 us.
struct SegmentPlan {
    int seg, hw;
};
inline SegmentPlan plan_segments(int64_t B, int64_t nc, int H, int P, int G) {
    const int items = H / G * ((P + kSlab - 1) / kSlab);
    for (int seg = 8; seg > 1; seg /= 2)
        for (int hw = items > 1 ? 2 : 1; hw > 0; --hw)
            if (nc > seg && B * ((nc + seg - 1) / seg) * G * ((items + hw - 1) / hw) >= 512) return {seg, hw};
    return {1, 1};
}

// Sections of the forward's workspace, which the backward reads again.  With segments the
// state of a segment's first chunk is what enters the segment, those of the others what its own
// tokens add to that, and `carried` and `decays`, the segments' decays, follow.
struct ScanWork {
    int nc, seg, hw;
    int64_t times, dt, shi, slo, decay, states, carried, decays, total;
};
inline ScanWork scan_work(int64_t B, int64_t L, int H, int P, int G, int N, bool bf16, bool save) {
    const int Q = 16 * (bf16 ? kStrips<bf16_t> : kStrips<float>);
    ScanWork w;
    w.nc = (int)((L + Q - 1) / Q);
    const SegmentPlan p = save ? SegmentPlan{1, 1} : plan_segments(B, w.nc, H, P, G);
    const int64_t state = (int64_t)P * state_cols(N), nseg = (w.nc + p.seg - 1) / p.seg;
    w.seg = p.seg;
    w.hw = p.hw;
    w.times = pad64(B * H * w.nc * Q);
    w.dt = 0;
    w.shi = w.times;
    w.slo = 2 * w.times;
    w.decay = 3 * w.times;
    w.states = w.decay + pad64(B * H * w.nc);
    w.carried = w.states + pad64(B * H * w.nc * state);
    w.decays = w.carried + (p.seg > 1 ? pad64(B * H * w.nc) : 0);
    w.total = w.decays + (p.seg > 1 ? pad64(B * H * nseg) : 0);
    return w;
}

// The chunks' own parts of the state (reverse: of the adjoint) into out [B, H, nc, P, cols].
template <typename T>
hipError_t launch_scan_states(const ScanDims &d, const T *X, int64_t x_batch, int64_t x_token, const T *Y,
                              int64_t y_batch, int64_t y_token, float *out, bool reverse, hipStream_t stream);
// The running states of segments (d.seg chunks, hw heads at once).
template <typename T>
hipError_t launch_scan_segments(const ScanDims &d, int hw, const T *X, int64_t x_batch, int64_t x_token, const T *Y,
                                int64_t y_batch, int64_t y_token, float *states, float *carried, float *decays,
                                hipStream_t stream);
// The recurrence over the chunks (or segments), in place; first / final [B, H, P, N] or null.
hipError_t launch_scan_pass(const ScanDims &d, float *states, const float *decays, const float *first, float *final_state,
                            int Q, bool reverse, hipStream_t stream);

// Runs X(NP, WHOLE) for the padded columns of the state and for P in whole vectors or not.
#define DDPM_SEQ_SCAN_SHAPES(T, N, P, X)             \
    if ((P) % kVec<T> == 0) {                        \
        if ((N) <= 32) X(32, true)                   \
        else if ((N) <= 64) X(64, true)              \
        else X(128, true)                            \
    } else {                                         \
        if ((N) <= 64) X(64, false)                  \
        else X(128, false)                           \
    }

}  // namespace seq
}  // namespace ddpm
