// Host-side declarations of the experts' kernels and the embedding lookup.
#pragma once

#include "aq_internal.h"

namespace aq {

// Arguments checked by the entry points.
struct RouteArgs {
    const aq_router *router;
    const void *x;
    int64_t T;
    int32_t *ids;
    float *weights;
    cudaStream_t stream;
};
cudaError_t moe_route_launch(const RouteArgs &a);

struct ExpertsArgs {
    const aq_experts *experts;
    int dtype;
    const void *x;
    int64_t T;
    int top_k;
    const int32_t *ids;
    const float *weights;
    void *out, *ws;
    cudaStream_t stream;
};
size_t moe_workspace_bytes(const aq_experts *x, int64_t T, int top_k);
cudaError_t moe_experts_launch(const ExpertsArgs &a);

cudaError_t embed_launch(int dtype, const void *ids, bool wide, int64_t T, const uint32_t *words,
                         const void *scales, const void *biases, int64_t N, int64_t K, int bits,
                         int group, float scale, void *out, cudaStream_t stream);

// One grid of the experts' products: PAIRS, the gate and up rows of every
// busy expert with SiLU (src: x in `dtype`, dst: h fp32 [T * top][R]);
// otherwise the down rows (src: h, dst: fp32 [T * top][R]).
struct MoeParams {
    const uint32_t *w0, *w1;
    const void *s0, *s1, *b0, *b1;  // fp16 scales and biases
    const int32_t *ids;
    const void *src;
    float *dst;
    int T, top, E, R, K, group, dtype;
};
cudaError_t moe_product_b2(const MoeParams &p, bool pairs, cudaStream_t stream);
cudaError_t moe_product_b3(const MoeParams &p, bool pairs, cudaStream_t stream);
cudaError_t moe_product_b4(const MoeParams &p, bool pairs, cudaStream_t stream);
cudaError_t moe_product_b5(const MoeParams &p, bool pairs, cudaStream_t stream);
cudaError_t moe_product_b6(const MoeParams &p, bool pairs, cudaStream_t stream);
cudaError_t moe_product_b8(const MoeParams &p, bool pairs, cudaStream_t stream);

// A launch whose grid may start while the stream's last one ends.
template <class P>
cudaError_t moe_launch(void (*kern)(P), dim3 grid, int threads, size_t smem, int cluster,
                       cudaStream_t stream, const P &prm) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, prm);
}

}  // namespace aq
