// aq_embed: rows of an affine-quantised table by token, out[t] = scale * (s q + b).
//
// The table is in the weight format (mlx-bun pages, @mlx-bun/inference 1.0.0,
// kernels/quantization/affine-split-mma.ts helper affine_unit), so a table
// that is also the vocabulary projection is kept once.  A thread takes 8
// values: B bytes of codes, which lie in two words at most, one 16-byte store.
// s q + b is one fp32 fma, the product with the scale one more rounding, the
// output type the last.  Four tokens' pieces are in flight a thread: 16,384
// rows of 4096 at 4 bits take 42 us (55 with one), 172 MB at 4.1 TB/s, three
// narrow loads behind the id's for each 16-byte store; a single token is a
// launch, 2 us.
#include "aq_moe.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace aq {
namespace {

struct EmbedParams {
    const void *ids;
    const uint32_t *words;
    const __half *scales, *biases;
    uint4 *out;
    int64_t T, N;
    int K, group, wide, bf16;
    float scale;
};

// 8 values of a row: the words of their codes, their scale and bias.
struct Piece {
    uint32_t w0, w1;
    __half s, b;
    bool live;
};

template <int B>
__device__ __forceinline__ Piece load_piece(const EmbedParams &p, int64_t id, int c) {
    Piece v = {0u, 0u, __half(0.f), __half(0.f), id >= 0 && id < p.N};
    if (v.live) {
        const int first = c * B / 4, sh = (c * B * 8) & 31;
        const uint32_t *row = p.words + id * (p.K * B / 32);
        v.w0 = row[first];
        if (sh + 8 * B > 32) v.w1 = row[first + 1];
        const int64_t at = id * (p.K / p.group) + c * 8 / p.group;
        v.s = p.scales[at];
        v.b = p.biases[at];
    }
    return v;
}

template <int B>
__device__ __forceinline__ uint4 decode_piece(const EmbedParams &p, const Piece &v, int c) {
    if (!v.live) return make_uint4(0u, 0u, 0u, 0u);
    const uint64_t codes = ((uint64_t)v.w1 << 32 | v.w0) >> ((c * B * 8) & 31);
    const float s = __half2float(v.s), b = __half2float(v.b);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float lo = fmaf(s, (float)((uint32_t)(codes >> (2 * j * B)) & ((1u << B) - 1u)), b) * p.scale;
        const float hi = fmaf(s, (float)((uint32_t)(codes >> ((2 * j + 1) * B)) & ((1u << B) - 1u)), b) * p.scale;
        if (p.bf16) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
            o[j] = *reinterpret_cast<const uint32_t *>(&x);
        } else {
            const __half2 x = __floats2half2_rn(lo, hi);
            o[j] = *reinterpret_cast<const uint32_t *>(&x);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// A block takes kRows tokens and a stretch of 8 * 256 columns: a thread has a
// piece of each token's row in flight at once.
constexpr int kRows = 4;
template <int B>
__global__ void __launch_bounds__(256) embed_kernel(const __grid_constant__ EmbedParams p) {
    const int per = p.K / 8;
    const int c = (int)blockIdx.y * 256 + (int)threadIdx.x;
    if (c >= per) return;
    const int64_t t0 = (int64_t)blockIdx.x * kRows;
    Piece v[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        int64_t id = -1;
        if (t0 + r < p.T)
            id = p.wide ? static_cast<const int64_t *>(p.ids)[t0 + r]
                        : (int64_t) static_cast<const int32_t *>(p.ids)[t0 + r];
        v[r] = load_piece<B>(p, id, c);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        if (t0 + r < p.T) p.out[(t0 + r) * per + c] = decode_piece<B>(p, v[r], c);
}

template <int B>
cudaError_t run(const EmbedParams &p, cudaStream_t stream) {
    const dim3 grid((unsigned)((p.T + kRows - 1) / kRows), (unsigned)((p.K / 8 + 255) / 256));
    embed_kernel<B><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t embed_launch(int dtype, const void *ids, bool wide, int64_t T, const uint32_t *words,
                         const void *scales, const void *biases, int64_t N, int64_t K, int bits,
                         int group, float scale, void *out, cudaStream_t stream) {
    const EmbedParams p = {ids, words, static_cast<const __half *>(scales),
                           static_cast<const __half *>(biases), static_cast<uint4 *>(out), T, N,
                           (int)K, group, wide ? 1 : 0, dtype == AQ_BF16 ? 1 : 0, scale};
    switch (bits) {
        case 2: return run<2>(p, stream);
        case 3: return run<3>(p, stream);
        case 4: return run<4>(p, stream);
        case 5: return run<5>(p, stream);
        case 6: return run<6>(p, stream);
        default: return run<8>(p, stream);
    }
}

}  // namespace aq
