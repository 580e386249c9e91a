// ff_launch.hip -- the feed-forward operators' products by type and kind, and the room they need.
#include <algorithm>

#include "ff_product.hpp"

namespace ddpm {
namespace ff {

#define DDPM_FF_KINDS(X) X(kForward, fwd) X(kGatedForward, gated) X(kGradX, gradx) X(kGradWeight, gradw)
#define X(K, name)                                                                    \
    hipError_t product_##name##_f32(const Product &a, void *work, hipStream_t stream); \
    hipError_t product_##name##_bf16(const Product &a, void *work, hipStream_t stream);
DDPM_FF_KINDS(X)
#undef X

hipError_t launch_product(Kind kind, const Product &a, void *work, bool bf16, hipStream_t stream) {
#define X(K, name) \
    if (kind == K) return bf16 ? product_##name##_bf16(a, work, stream) : product_##name##_f32(a, work, stream);
    DDPM_FF_KINDS(X)
#undef X
    return hipErrorInvalidValue;
}

template <typename T>
static int64_t bytes_of(Kind kind, int64_t np, int64_t nq, int64_t nk, int terms) {
    int64_t most = 0;
    for (const bool direct : {false, true}) {
        if (few_rows(kind, np, nq, nk, Elem<T>::is_bf16, direct)) continue;
        most = std::max(most, part_bytes(Elem<T>::is_bf16, kind, cut_of<T>(kind, np, nq, nk, terms, direct)));
    }
    return most;
}

int64_t product_bytes(Kind kind, int64_t np, int64_t nq, int64_t nk, int terms, bool bf16) {
    return bf16 ? bytes_of<bf16_t>(kind, np, nq, nk, terms) : bytes_of<float>(kind, np, nq, nk, terms);
}

double product_time(Kind kind, int64_t np, int64_t nq, int64_t nk, int terms, bool bf16, bool straight) {
    const double t = bf16 ? cut_of<bf16_t>(kind, np, nq, nk, terms, straight).cost : cut_of<float>(kind, np, nq, nk, terms, straight).cost;
    // The form for any alignment takes 1.7 times as long with both operands along their rows, and 3.3 and
    // 5.5 times with one and both read by columns (bfloat16, products of 4095^3; float32 1.1 to 1.4).
    return straight ? t : t * (!bf16 ? 1.25 : kind == kGradX ? 3.3 : kind == kGradWeight ? 5.5 : 1.7);
}

double copies_time(int64_t bytes) { return 5. + 2. * (double)bytes / kBytes; }

}  // namespace ff
}  // namespace ddpm
