// ff_gated_f32.hip -- one kind of the feed-forward operators' products (ff_gemm.hpp).
#include "ff_product.hpp"

namespace ddpm {
namespace ff {

hipError_t product_gated_f32(const Product &a, void *work, hipStream_t stream) { return product<float, kGatedForward>(a, work, stream); }

}  // namespace ff
}  // namespace ddpm
