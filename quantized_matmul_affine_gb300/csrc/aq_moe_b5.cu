// The experts' products with 5-bit codes (a translation unit a width, so that
// they compile in parallel).
#include "aq_moe.cuh"

namespace aq {

cudaError_t moe_product_b5(const MoeParams &p, bool pairs, int variant, cudaStream_t stream) {
    return moe_detail::launch<5>(p, pairs, variant, stream);
}

cudaError_t moe_pack_b5(const MoeParams &p, bool pairs, uint8_t *to, cudaStream_t stream) {
    return moe_detail::pack<5>(p, pairs, to, stream);
}

}  // namespace aq
