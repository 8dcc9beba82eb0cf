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
    const uint8_t *packed;  // the source rows as the MMA wants them (MoePack), or null
};
// The products' kernels: columns (tokens of an expert) taken at a time, and
// whether they come from packed rows.
enum MoeVariant { MOE_8 = 0, MOE_8_PACKED, MOE_16, MOE_32 };
inline bool moe_packed(int variant) { return variant >= MOE_8_PACKED; }

// Packed source rows: [rows][K] fp16 in MMA order, then the group sums, 16 bytes
// of either part a block of 8 groups (4 of 128 and zeros), then the inverse
// powers of two, floats, each part 256-byte aligned.
struct MoePack {
    int64_t sums, undo, bytes;  // byte offsets, and the whole
    int blocks;                 // a row's
};
#ifdef __CUDACC__
__host__ __device__
#endif
inline MoePack moe_pack(int64_t rows, int64_t K, int group) {
    MoePack m;
    m.blocks = (int)((K / (group == 32 ? 256 : 512)) + (K % (group == 32 ? 256 : 512) != 0));
    m.sums = (rows * K * 2 + 255) & ~(int64_t)255;
    m.undo = m.sums + ((rows * m.blocks * 32 + 255) & ~(int64_t)255);
    m.bytes = m.undo + ((rows * 4 + 255) & ~(int64_t)255);
    return m;
}
// Packs rows of p.src (PAIRS as above: x, T rows, or h, T * top) to `to`.
cudaError_t moe_pack_b2(const MoeParams &p, bool pairs, uint8_t *to, cudaStream_t stream);
cudaError_t moe_pack_b3(const MoeParams &p, bool pairs, uint8_t *to, cudaStream_t stream);
cudaError_t moe_pack_b4(const MoeParams &p, bool pairs, uint8_t *to, cudaStream_t stream);
cudaError_t moe_pack_b5(const MoeParams &p, bool pairs, uint8_t *to, cudaStream_t stream);
cudaError_t moe_pack_b6(const MoeParams &p, bool pairs, uint8_t *to, cudaStream_t stream);
cudaError_t moe_pack_b8(const MoeParams &p, bool pairs, uint8_t *to, cudaStream_t stream);
cudaError_t moe_product_b2(const MoeParams &p, bool pairs, int variant, cudaStream_t stream);
cudaError_t moe_product_b3(const MoeParams &p, bool pairs, int variant, cudaStream_t stream);
cudaError_t moe_product_b4(const MoeParams &p, bool pairs, int variant, cudaStream_t stream);
cudaError_t moe_product_b5(const MoeParams &p, bool pairs, int variant, cudaStream_t stream);
cudaError_t moe_product_b6(const MoeParams &p, bool pairs, int variant, cudaStream_t stream);
cudaError_t moe_product_b8(const MoeParams &p, bool pairs, int variant, cudaStream_t stream);

// A launch whose grid may start while the stream's last one ends.
template <class... P, class... A>
cudaError_t moe_launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, int cluster,
                       cudaStream_t stream, A... prm) {
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
    return cudaLaunchKernelEx(&cfg, kern, prm...);
}

}  // namespace aq
