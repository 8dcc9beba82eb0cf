// The experts' products with 4-bit codes (a translation unit a width, so that
// they compile in parallel).
#include "aq_moe.cuh"

namespace aq {

cudaError_t moe_product_b4(const MoeParams &p, bool pairs, cudaStream_t stream) {
    return moe_detail::launch<4>(p, pairs, stream);
}

}  // namespace aq
