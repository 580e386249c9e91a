// ff_launch.hip -- the feed-forward operators' products by type and kind.
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

}  // namespace ff
}  // namespace ddpm
