// ff_launch.hip -- the feed-forward operators' products by type and kind, and the room they need.
#include <algorithm>

#include "ff_product.hpp"

namespace ddpm {
namespace ff {

#define DDPM_FF_KINDS(X) X(kForward, fwd) X(kGatedForward, gated) X(kGradX, gradx) X(kGradWeight, gradw)
#define X(K, name)                                                                    \
    hipError_t product_##name##_f32(const Product &a, float *part, hipStream_t stream); \
    hipError_t product_##name##_bf16(const Product &a, float *part, hipStream_t stream);
DDPM_FF_KINDS(X)
#undef X

hipError_t launch_product(Kind kind, const Product &a, float *part, bool bf16, hipStream_t stream) {
#define X(K, name) \
    if (kind == K) return bf16 ? product_##name##_bf16(a, part, stream) : product_##name##_f32(a, part, stream);
    DDPM_FF_KINDS(X)
#undef X
    return hipErrorInvalidValue;
}

int64_t product_floats(Kind kind, int64_t np, int64_t nq, int64_t nk, bool bf16) {
    int64_t most = 0;
    for (const bool direct : {false, true}) {
        if (few_rows(kind, nq, direct)) continue;
        const Cut c = bf16 ? cut_of<bf16_t>(kind, np, nq, nk, direct) : cut_of<float>(kind, np, nq, nk, direct);
        most = std::max(most, c.pieces > 1 ? part_floats(bf16, kind, c) : 0);
    }
    return most;
}

}  // namespace ff
}  // namespace ddpm
