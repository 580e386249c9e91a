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
// the same.  float32: 64, since its matrix products cost 16 times as much.
template <typename T> constexpr int kStrips = Elem<T>::is_bf16 ? 8 : 4;

struct ScanDims {
    int B, L, H, P, G, N, nc;  // nc: chunks
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
// share B and C: a workgroup takes as many as still leave `target` workgroups.
inline ChunkPlan plan_heads(int64_t B, int64_t nc, int H, int G, int64_t target) {
    const int64_t base = B * nc * G;
    const int hg = H / G;
    int64_t splits = (target + base - 1) / base;
    if (splits > hg) splits = hg;
    const int per = (int)((hg + splits - 1) / splits);
    return {per, (hg + per - 1) / per};
}

__device__ __forceinline__ int valid_tokens(const int *lengths, int b, int L) {
    if (lengths == nullptr) return L;
    const int n = lengths[b];
    return n < 0 ? 0 : n > L ? L : n;
}

inline int64_t pad64(int64_t n) { return (n + 63) / 64 * 64; }

// Sections of the forward's workspace, which the backward reads again.
struct ScanWork {
    int nc;
    int64_t times, dt, shi, slo, decay, states, total;
};
inline ScanWork scan_work(int64_t B, int64_t L, int H, int P, int N, int Q) {
    ScanWork w;
    w.nc = (int)((L + Q - 1) / Q);
    w.times = pad64(B * H * w.nc * Q);
    w.dt = 0;
    w.shi = w.times;
    w.slo = 2 * w.times;
    w.decay = 3 * w.times;
    w.states = w.decay + pad64(B * H * w.nc);
    w.total = w.states + pad64(B * H * w.nc * (int64_t)P * state_cols(N));
    return w;
}

// The chunks' own parts of the state (reverse: of the adjoint) into out [B, H, nc, P, cols].
template <typename T>
hipError_t launch_scan_states(const ScanDims &d, const T *X, int64_t x_batch, int64_t x_token, const T *Y,
                              int64_t y_batch, int64_t y_token, float *out, bool reverse, hipStream_t stream);
// The recurrence over the chunks, in place; first / final [B, H, P, N] or null.
hipError_t launch_scan_pass(const ScanDims &d, float *states, const float *first, float *final_state, int Q,
                            bool reverse, hipStream_t stream);

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
