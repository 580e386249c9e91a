// ff_launch.hpp -- kernel launchers of the feed-forward operators.  They check nothing but grid
// limits (hipErrorInvalidConfiguration); arguments are validated in ff_abi.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ff_plan.hpp"

namespace ddpm {
namespace ff {

// out[q][p] = sum over k < nk of P(p, k) Q(q, k), out [nq, np] contiguous; the gated product has np
// columns and 2 np rows of P.  Strides in elements.
struct Product {
    const void *p, *q;
    int64_t p_ld, q_ld, np, nq, nk;
    bool p_padded, q_padded;            // rows that end in zeros up to whole 16-byte chunks
    int64_t low;                        // gradients: elements from Q to its second term (two_terms), or 0
    void *out;
    void *sums;                         // weight's gradient: [nq], sums over k of Q
    float *saved;                       // forward: what the activation is applied to, or null
    const void *bias, *residual;        // forward: or null
    int64_t residual_ld;
    int act;
    // Where the backward makes z again: the forward writes its bias here in float32, and the backward's
    // call has it with grad [nq, np], and out is dz (rows and terms, `low` apart, as launch_dz writes them).
    float *kept;
    const void *grad;
    int64_t grad_ld;
    // The first `whole` of tiles_p * tiles_q tiles are a workgroup's each; the others are cut along the
    // contraction into `pieces` of `run` elements, whose results go to `part` in float32.
    uint32_t tiles_p, tiles_q, whole;
    int pieces;
    int64_t run;
    float *part;
};

hipError_t launch_product(Kind kind, const Product &a, void *work, bool bf16, hipStream_t stream);

// A copy of an operand whose rows would otherwise start anywhere: rows of whole lines (padded), their last 16-byte chunk
// filled up with zeros.
struct Copy {
    const void *src;
    int64_t ld, rows, cols;
    void *dst;  // [rows, padded(cols)]; 16-byte aligned
};
// One or two copies; the second may have no rows.
hipError_t launch_copies(const Copy &a, const Copy &b, bool bf16, hipStream_t stream);

// The forward products of few rows (ff_rows.hip), from operands that can go straight to LDS (chunked) or from any.
hipError_t launch_rows(bool gated, bool chunked, const Product &a, bool bf16, hipStream_t stream);

// dz = grad * act'(saved), [rows, N]; gated: saved [rows, 2 N] and dz [rows, 2 N],
// the gate's half grad * u * act'(g), the other grad * act(g).
// dz's rows are padded as a Copy's; its second term, what rounding the first one left, is `low` elements behind
// it (0: one term).
hipError_t launch_dz(bool gated, const void *grad, int64_t grad_ld, const float *saved, void *dz, int64_t low, int64_t rows,
                     int64_t N, int act, bool bf16, hipStream_t stream);

// The whole backward through an activation or a gate of few channels, which makes z again
// (ff_small.hip).
struct SmallBackward {
    const void *grad, *x, *weight;
    const float *bias;                  // [N], gated [2 N]
    int64_t rows, grad_ld, x_ld, weight_ld;
    int C, N, act;
    void *grad_x;                       // [rows, C] or null
    float *part;                        // of grad_weight and grad_bias, or null with them
};
hipError_t launch_small_backward(bool gated, SmallBackward a, void *grad_weight, void *grad_bias, bool bf16, hipStream_t stream);

}  // namespace ff
}  // namespace ddpm
