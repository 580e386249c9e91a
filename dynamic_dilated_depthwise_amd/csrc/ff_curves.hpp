// ff_curves.hpp -- the activations of the feed-forward operators and their derivatives, in float32, to
// a few roundings (8 at most for gelu, below zero too) and without branches: in the epilogue of a large
// tile all waves are in them at once (gelu from the library's erfc took as long as sixteen steps of
// the contraction).
//
//   silu  z s,  s = 1 / (1 + exp(-z));        derivative s (1 + z (1 - s))
//   gelu  z Phi(z);                           derivative Phi(z) + z phi(z)
//
// Phi below zero is phi's exponential times the scaled complementary error function, which is t times
// a polynomial of degree 9 in t = 1 / (1 + 0.45 |z| / sqrt 2) (least squares over the whole half line,
// weighted to equal relative errors of 3.2e-8).
#pragma once

#include "../../include/ddpm_ff.h"
#include "common.hpp"

namespace ddpm {
namespace ff {

constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;

// exp(-z); z is limited so that the exponent stays a number (the results are 0 or infinite long before).
__device__ __forceinline__ float exp_minus(float z) {
    const float v = fminf(fmaxf(z, -200.f), 200.f), a = v * -kLog2e;
    const float rest = fmaf(v, -kLog2e, -a) - v * 1.92596299e-8f;  // what a lost, and log2(e)'s own rest
    return __builtin_amdgcn_exp2f(a) * fmaf(rest, kLn2, 1.f);
}
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + exp_minus(z)); }

// Phi(z) and exp(-z^2 / 2).
struct Normal {
    float below, bell;
};
__device__ __forceinline__ Normal normal(float z) {
    const float v = fminf(fabsf(z), 19.8f), s = v * v;  // exp(-19.8^2 / 2) is 0
    const float a = s * (-0.5f * kLog2e), rest = fmaf(fmaf(v, v, -s), -0.5f * kLog2e, fmaf(s, -0.5f * kLog2e, -a)) - s * 9.62981496e-9f;
    const float bell = __builtin_amdgcn_exp2f(a) * fmaf(rest, kLn2, 1.f);
    const float t = __builtin_amdgcn_rcpf(fmaf(v, 0.45f * 0.70710678f, 1.f));
    float p = -2.069557831e-02f;
    p = fmaf(p, t, 9.534404427e-02f);
    p = fmaf(p, t, -1.502913982e-01f);
    p = fmaf(p, t, 7.120060176e-02f);
    p = fmaf(p, t, -1.117901690e-02f);
    p = fmaf(p, t, 5.997522548e-02f);
    p = fmaf(p, t, 8.762606233e-02f);
    p = fmaf(p, t, 1.141358241e-01f);
    p = fmaf(p, t, 1.269415766e-01f);
    p = fmaf(p, t, 1.269426644e-01f);
    const float q = bell * (p * t);
    return {z < 0.f ? q : 1.f - q, bell};
}

template <int ACT> __device__ __forceinline__ float curve_of(float z) {
    if constexpr (ACT == DDPM_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays
    else if constexpr (ACT == DDPM_ACT_SILU) return z * sigmoid(z);
    else if constexpr (ACT == DDPM_ACT_GELU) return z * normal(z).below;
    else return z;
}
// The activation and its derivative.
template <int ACT> __device__ __forceinline__ void curve_and_slope(float z, float &a, float &d) {
    if constexpr (ACT == DDPM_ACT_RELU) {
        a = curve_of<ACT>(z);
        d = z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
    } else if constexpr (ACT == DDPM_ACT_SILU) {
        const float s = sigmoid(z);
        a = z * s;
        d = s * fmaf(z, 1.f - s, 1.f);
    } else if constexpr (ACT == DDPM_ACT_GELU) {
        const Normal n = normal(z);
        a = z * n.below;
        d = fmaf(z * 0.39894228f, n.bell, n.below);
    } else {
        a = z;
        d = 1.f;
    }
}

// v = act(v), the choice outside the loop.
__device__ __forceinline__ void activate(float (&v)[8], int act) {
#define X(ACT)                                              \
    if (act == ACT) {                                       \
        _Pragma("unroll") for (int e = 0; e < 8; ++e) v[e] = curve_of<ACT>(v[e]); \
    }
    X(DDPM_ACT_RELU) else X(DDPM_ACT_SILU) else X(DDPM_ACT_GELU)
#undef X
}
// a = act(z), d = act'(z).
template <int n>
__device__ __forceinline__ void slopes(const float (&z)[n], float (&a)[n], float (&d)[n], int act) {
#define X(ACT)                                              \
    if (act == ACT) {                                       \
        _Pragma("unroll") for (int e = 0; e < n; ++e) curve_and_slope<ACT>(z[e], a[e], d[e]); \
    }
    X(DDPM_ACT_NONE) else X(DDPM_ACT_RELU) else X(DDPM_ACT_SILU) else X(DDPM_ACT_GELU)
#undef X
}

}  // namespace ff
}  // namespace ddpm
