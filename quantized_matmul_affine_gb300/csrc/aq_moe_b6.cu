// The experts' products with 6-bit codes (a translation unit a width, so that
// they compile in parallel).
#include "aq_moe.cuh"

namespace aq {

cudaError_t moe_product_b6(const MoeParams &p, bool pairs, cudaStream_t stream) {
    return moe_detail::launch<6>(p, pairs, stream);
}

}  // namespace aq
