// ff_gradx_bf16.hip -- one kind of the feed-forward operators' products (ff_gemm.hpp).
#include "ff_product.hpp"

namespace ddpm {
namespace ff {

hipError_t product_gradx_bf16(const Product &a, void *work, hipStream_t stream) { return product<bf16_t, kGradX>(a, work, stream); }

}  // namespace ff
}  // namespace ddpm
