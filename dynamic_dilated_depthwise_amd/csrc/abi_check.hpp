// abi_check.hpp -- argument checks that the operators' C entry points share: sizes, strides, pointers,
// and outputs that overlap.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ddpm.h"

namespace ddpm {
namespace abi {

constexpr int64_t kMax = 0x7fffffff;
constexpr int64_t kMaxRun = kMax - 65535;  // of what kernels walk: the end of a last, partial block stays an int
constexpr double kMostElements = 1e17;  // of a tensor: keeps every product of sizes in 64 bits

struct Span {
    const void *p;
    double bytes;
};

// Collects a call's arguments; `bad` once any of them is wrong.
struct Check {
    int dtype;
    bool bad = false;
    Span in[16], out[16];
    int ins = 0, outs = 0;

    explicit Check(int dt) : dtype(dt), bad(dt != DDPM_F32 && dt != DDPM_BF16) {}
    int64_t es() const { return dtype == DDPM_BF16 ? 2 : 4; }
    void size(int64_t v, int64_t most = kMax) { bad |= v < 1 || v > most; }
    void stride(int64_t v) { bad |= v < 0 || v > (int64_t(1) << 46); }
    void pointer(const void *p, int64_t align) { bad |= p == nullptr || (uintptr_t)p % align != 0; }
    void input(const void *p, double count, int64_t width) {
        pointer(p, width);
        in[ins++] = {p, count * width};
    }
    void output(const void *p, double count, int64_t width) {
        pointer(p, width);
        out[outs++] = {p, count * width};
    }
    void maybe_in(const void *p, double count, int64_t width) {
        if (p != nullptr) input(p, count, width);
    }
    void maybe_out(const void *p, double count, int64_t width) {
        if (p != nullptr) output(p, count, width);
    }
    void workspace(const void *p, double bytes) {
        pointer(p, 16);
        out[outs++] = {p, bytes};
    }
    int done() {
        for (int i = 0; i < outs && !bad; ++i) {
            if (out[i].bytes > 9.0e18) bad = true;
            for (int k = 0; k < ins; ++k) bad |= overlap(out[i], in[k]);
            for (int k = 0; k < i; ++k) bad |= overlap(out[i], out[k]);
        }
        return bad ? DDPM_ERR_INVALID_ARG : DDPM_OK;
    }
    static bool overlap(const Span &a, const Span &b) {
        const double a0 = (double)(uintptr_t)a.p, b0 = (double)(uintptr_t)b.p;
        if (a0 != b0) return a0 < b0 ? a0 + a.bytes > b0 : b0 + b.bytes > a0;
        return a.bytes > 0 && b.bytes > 0;
    }
};

// Elements between the first and the last of a [batch, length, row] view.
inline double extent(int64_t batch, int64_t length, int64_t row, int64_t sb, int64_t st) {
    return (double)(batch - 1) * sb + (double)(length - 1) * st + row;
}

inline int status_of(hipError_t e) {
    if (e == hipSuccess) return DDPM_OK;
    return e == hipErrorInvalidConfiguration ? DDPM_ERR_UNSUPPORTED : DDPM_ERR_HIP;
}

inline bool is_bf16(int dtype) { return dtype == DDPM_BF16; }

}  // namespace abi
}  // namespace ddpm
