// The experts' products with 2-bit codes (a translation unit a width, so that
// they compile in parallel).
#include "aq_moe.cuh"

namespace aq {

cudaError_t moe_product_b2(const MoeParams &p, bool pairs, int variant, cudaStream_t stream) {
    return moe_detail::launch<2>(p, pairs, variant, stream);
}

cudaError_t moe_pack_b2(const MoeParams &p, bool pairs, uint8_t *to, cudaStream_t stream) {
    return moe_detail::pack<2>(p, pairs, to, stream);
}

}  // namespace aq
