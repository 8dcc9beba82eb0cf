// The experts' products of a mixture-of-experts layer for few tokens: for
// every expert that some token picked, its affine rows times those tokens'
// activations, on warp MMA.
//
//   gate and up:  h[t,j][i] = silu(g) * u,  g = Wg_e[i] . x[t],  u = Wu_e[i] . x[t]
//   down:         d[t,j][n] = Wd_e[n] . h[t,j]              with e = ids[t][j]
//
// in the factored form of the affine kernels (mlx-bun pages,
// @mlx-bun/inference 1.0.0, kernels/quantization/affine4-rows.ts and
// affine3-rows.ts headers): per group, scale * sum(q x) + bias * sum(x).
//
//   * Work is the list of 16-row MMA tiles (8 gate and the same 8 up rows, or
//     16 down rows) of all busy experts, in expert order, dealt to the CTAs in
//     runs of even cost.  A CTA takes its run expert by expert; an expert's tiles
//     go round the 8 warps, and the last, unfull round's tiles are shared by 2, 4
//     or 8 warps that split K and add their parts in order: the result does not
//     depend on timing.
//   * A warp streams its tiles by itself: three steps of 128 values of K, 64
//     bytes of 16 rows each at 4 bits, are on their way to its own ring in shared
//     memory by asynchronous copies, with the blocks of scales they need, and the
//     next tile's follow without a stop.  Lane (g, q) of the MMA layout reads the
//     16 codes [16q, 16q + 16) of rows g and g + 8 of a unit.  The MMA's k order
//     within a unit is whatever the decode gives (Order): the activations are
//     staged, or packed, in that order.
//   * A code masked in place in an fp16 with zero exponent is the exact
//     subnormal q * 2^(p - 24), p its bit position; the activation paired with
//     it carries 2^-p (p is 8 at most at 2 bits, 6 at 3, 5 at 5, 4 at 4, 0 at 6
//     and 8; with groups of 32 also 6 at 2).  Activations are fp16 with one power
//     of two per token that puts the row's largest magnitude into [2^14, 2^15):
//     bf16 and fp16 values above 2^(p - 28) of it keep all their bits, smaller
//     ones are off by 2^(p - 39) of it at most (which shows only where the
//     weights of all large values are near zero); h (fp32) is rounded to fp16's
//     11 bits, 2^-11 of a value at most, an eighth of what rounding it to bf16
//     would cost.  Sums of codes, group sums and everything after them are fp32.
//   * The biases enter as products of their own, 8 groups a step, with the
//     columns' group sums, which are kept as two fp16 parts: 22 bits, down to
//     2^-31 of the row's largest magnitude.
//   * Tokens of an expert are MMA columns, 8, 16 or 32 at a time; blocks of 8
//     that are empty are skipped.  An expert with more takes its weights again,
//     from L2.
//
// Where the experts are large, bound by the copies into shared memory: 8
// experts of 4096 x 13824 at 4 bits (688 MB) take 205 us a layer; gate and up 114
// of them and down 74, 4.0 and 3.1 TB/s; with the arithmetic left out 190 us, so
// it is nearly hidden; with the codes left out 68 us, and with the loop left out
// 44 us (six dependent launches, plans, staged columns).  What limits the codes is
// how they are copied, 16 bytes a lane with an address and a predicate each.  For
// one token the kernels' starts are all there is (128 experts of 2048 x 768: 28
// us for 22 MB).  24 warps of up to 80 registers an SM: 16 warps of 128 with two tiles a
// step were as fast on large runs and slower on short ones.
#pragma once

#include "aq_moe.h"
#include "aq_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

namespace aq {
namespace moe_detail {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr uint16_t kNone = 0xFFFF;
constexpr int kMaxEntries = AQ_MOE_MAX_TOKENS * AQ_MOE_MAX_TOP;

// A lane's 16 codes of one row and unit are codes [16q, 16q + 16), or with
// groups of 32 codes [8q, 8q + 8) of either group, so that the MMA's first two
// k steps are one group and the last two the other.  Order says how they land
// in 8 registers of fp16 pairs: register p holds codes lo(p) and hi(p) of the
// lane's 16, at bit position pre(p).
template <int B, bool G32>
struct Order {
    static constexpr int kHalf = G32 ? 4 : 8;  // distance of a pair's codes in the odd widths
    __host__ __device__ static constexpr int lo(int p) {
        return B == 4 ? (p / 4) * 8 + p % 4 : B == 8 ? (p / 2) * 4 + p % 2 : (p / kHalf) * 8 + p % kHalf;
    }
    __host__ __device__ static constexpr int hi(int p) {
        return lo(p) + (B == 4 ? 4 : B == 8 ? 2 : kHalf);
    }
    __host__ __device__ static constexpr int pre(int p) {
        const int k = p % kHalf;
        return B == 2   ? (k < 5 ? 2 * k : 2 * (k - 5))
               : B == 3 ? (k < 3 ? 3 * k : k < 5 ? 3 * (k - 3) : 3 * (k - 5))
               : B == 4 ? 4 * (p & 1)
               : B == 5 ? (k % 3 == 1 ? 5 : 0)
                        : 0;
    }
};

// 32-bit words that hold a lane's 16 codes (codes that start or end inside a
// word bring their neighbours along).
template <int B, bool G32>
constexpr int kWords = B == 8 ? 4 : B == 4 ? 2 : G32 ? (B == 2 ? 2 : 4) : (B == 2 ? 1 : B == 3 ? 2 : 3);
// Units of 64 values taken in one step: two where that makes a row's codes of
// a step whole 16-byte pieces.
template <int B>
constexpr int kUnits = B == 6 || B == 8 ? 1 : 2;

// First bit of the lane's codes in a unit's row (with groups of 32 the second
// group's lie B words on).
template <int B, bool G32>
__device__ __forceinline__ int first_bit(int q) {
    return (G32 ? 8 : 16) * B * q;
}

// Shared memory by 32-bit address: the loop's addresses stay in one register.
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
template <int N>
__device__ __forceinline__ void lds(uint32_t a, uint32_t *v) {
    if constexpr (N == 4) {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(a)
                     : "memory");
    } else if constexpr (N == 2) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a) : "memory");
    } else {
        static_assert(N == 1, "1, 2 or 4 words");
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(a) : "memory");
    }
}

// The words of a lane's codes of one row and unit.
template <int B, bool G32>
__device__ __forceinline__ void load_codes(uint32_t a, uint32_t (&w)[kWords<B, G32>]) {
    constexpr int N = kWords<B, G32>;
    if constexpr (!G32 && (B == 4 || B == 8)) {
        lds<N>(a, w);
    } else if constexpr (!G32) {
#pragma unroll
        for (int i = 0; i < N; ++i) lds<1>(a + 4 * i, w + i);
    } else if constexpr (B == 8) {
        lds<2>(a, w);
        lds<2>(a + 32, w + 2);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < N / 2; ++i) lds<1>(a + 4 * (B * h + i), w + h * (N / 2) + i);
    }
}

// A lane's 16 codes as 8 registers of two fp16 subnormals each; sh: where they
// start in the first word.
template <int B, bool G32>
__device__ __forceinline__ void decode(const uint32_t (&w)[kWords<B, G32>], uint32_t sh,
                                       uint32_t (&r)[8]) {
    if constexpr (B == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t v = w[i] >> 8;
            r[4 * i] = w[i] & 0x000F000Fu;
            r[4 * i + 1] = w[i] & 0x00F000F0u;
            r[4 * i + 2] = v & 0x000F000Fu;
            r[4 * i + 3] = v & 0x00F000F0u;
        }
    } else if constexpr (B == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[2 * i] = w[i] & 0x00FF00FFu;
            r[2 * i + 1] = prmt(w[i], 0u, 0x4341u);  // bytes 1 and 3
        }
    } else if constexpr (G32) {
        // 8 codes of each group: the first four and the last four side by side
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t *o = r + 4 * h;
            if constexpr (B == 2) {
                const uint32_t a = w[h] >> sh, x = prmt(a, a >> 8, 0x5410u);
                o[0] = x & 0x00030003u;
                o[1] = x & 0x000C000Cu;
                o[2] = x & 0x00300030u;
                o[3] = x & 0x00C000C0u;
            } else {
                const uint32_t a = __funnelshift_r(w[2 * h], w[2 * h + 1], sh);
                if constexpr (B == 3) {
                    const uint32_t x = prmt(a, a >> 12, 0x5410u);
                    o[0] = x & 0x00070007u;
                    o[1] = x & 0x00380038u;
                    o[2] = x & 0x01C001C0u;
                    o[3] = (x >> 9) & 0x00070007u;
                } else {
                    const uint32_t b = w[2 * h + 1] >> sh;
                    const uint32_t t = __funnelshift_r(a, b, 4 * B);
                    uint32_t x = prmt(a, t, 0x5410u);
                    if constexpr (B == 5) {
                        o[0] = x & 0x001F001Fu;
                        o[1] = x & 0x03E003E0u;
                        o[2] = (x >> 10) & 0x001F001Fu;
                        o[3] = prmt(a >> 15, t >> 15, 0x5410u) & 0x001F001Fu;
                    } else {
                        o[0] = x & 0x003F003Fu;
                        o[1] = (x >> 6) & 0x003F003Fu;
                        x = prmt(a >> 12, t >> 12, 0x5410u);
                        o[2] = x & 0x003F003Fu;
                        o[3] = (x >> 6) & 0x003F003Fu;
                    }
                }
            }
        }
    } else if constexpr (B == 2) {
        const uint32_t v = w[0] >> 10;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            r[j] = j < 5 ? w[0] & (0x00030003u << (2 * j)) : v & (0x00030003u << (2 * (j - 5)));
    } else if constexpr (B == 3) {
        // the halves of the 48 bits, 24 each, side by side
        const uint32_t a = __funnelshift_r(w[0], w[1], sh), b = w[1] >> sh;
        const uint32_t t = __funnelshift_r(a, b, 24);
        const uint32_t p = prmt(a, t, 0x5410u), v = p >> 9, u = prmt(a >> 15, t >> 15, 0x5410u);
        r[0] = p & 0x00070007u;
        r[1] = p & 0x00380038u;
        r[2] = p & 0x01C001C0u;
        r[3] = v & 0x00070007u;
        r[4] = v & 0x00380038u;
        r[5] = u & 0x00070007u;
        r[6] = u & 0x00380038u;
        r[7] = u & 0x01C001C0u;
    } else if constexpr (B == 5) {
        const uint32_t a0 = __funnelshift_r(w[0], w[1], sh), a1 = __funnelshift_r(w[1], w[2], sh);
        const uint32_t a2 = w[2] >> sh;
        const uint32_t t0 = __funnelshift_r(a1, a2, 8), t1 = a2 >> 8;
        uint32_t x = prmt(a0, t0, 0x5410u);
        r[0] = x & 0x001F001Fu;
        r[1] = x & 0x03E003E0u;
        r[2] = (x >> 10) & 0x001F001Fu;
        x = prmt(a0 >> 15, t0 >> 15, 0x5410u);
        r[3] = x & 0x001F001Fu;
        r[4] = x & 0x03E003E0u;
        r[5] = (x >> 10) & 0x001F001Fu;
        x = prmt(__funnelshift_r(a0, a1, 30), __funnelshift_r(t0, t1, 30), 0x5410u);
        r[6] = x & 0x001F001Fu;
        r[7] = x & 0x03E003E0u;
    } else {
        static_assert(B == 6, "2, 3, 4, 5, 6 or 8 bits");
        const uint32_t t0 = __funnelshift_r(w[1], w[2], 16), t1 = w[2] >> 16;
        uint32_t x = prmt(w[0], t0, 0x5410u);
        r[0] = x & 0x003F003Fu;
        r[1] = (x >> 6) & 0x003F003Fu;
        x = prmt(w[0] >> 12, t0 >> 12, 0x5410u);
        r[2] = x & 0x003F003Fu;
        r[3] = (x >> 6) & 0x003F003Fu;
        x = prmt(__funnelshift_r(w[0], w[1], 24), __funnelshift_r(t0, t1, 24), 0x5410u);
        r[4] = x & 0x003F003Fu;
        r[5] = (x >> 6) & 0x003F003Fu;
        x = prmt(w[1] >> 4, t1 >> 4, 0x5410u);
        r[6] = x & 0x003F003Fu;
        r[7] = (x >> 6) & 0x003F003Fu;
    }
}

// d = a b + d, or without d.
__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                     uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(b0));
}

// The words of 8 source values, from x (fp16 or bf16) or h (fp32); ordinary
// loads, since this grid may have started before they were written.
template <bool PAIRS>
__device__ __forceinline__ void source8(const MoeParams &p, size_t at, uint32_t *w) {
    const uint8_t *s = static_cast<const uint8_t *>(p.src) + at * (PAIRS ? 2 : 4);
#pragma unroll
    for (int i = 0; i < (PAIRS ? 1 : 2); ++i)
        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                     : "l"(s + 16 * i)
                     : "memory");
}
template <bool PAIRS>
__device__ __forceinline__ void widen16(const MoeParams &p, const uint32_t (&w)[PAIRS ? 8 : 16], float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if constexpr (!PAIRS) {
            v[i] = __uint_as_float(w[i]);
        } else if (p.dtype == AQ_BF16) {
            v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        } else {
            const __half2 h = *reinterpret_cast<const __half2 *>(&w[i / 2]);
            v[i] = i & 1 ? __high2float(h) : __low2float(h);
        }
    }
}

struct Shared {
    int count[AQ_MOE_MAX_EXPERTS];     // entries of each expert
    int before[AQ_MOE_MAX_EXPERTS];    // cost of a tile of the busy experts before each
    uint16_t act[AQ_MOE_MAX_EXPERTS];  // the busy experts, ascending
    uint16_t list[32];                 // entries t * top + j of the current columns
    uint32_t peak[32];                 // a column's largest magnitude, as bits
    float undo[32];                    // a column's inverse power of two
    int warp_sum[kWarps];
    int busy, cost;
};
// Dynamic shared memory of a CTA, n of them an SM.
constexpr int dynamic_bytes(int n) { return (228 * 1024 / n - 1024 - (int)sizeof(Shared)) & ~127; }

// What a tile of an expert with n entries costs, in columns' products: the
// codes are decoded once for every C columns, as much work as about four
// products with 8 columns.
template <int C>
__device__ __forceinline__ int tile_cost(int n) {
    return 4 * ((n + C - 1) / C) + (n + 7) / 8;
}

// Counts the entries of every expert, lists the busy experts in order with the
// costs before them, and keeps every entry's expert in ids (kNone without one).
template <int C>
__device__ __forceinline__ void plan(const MoeParams &p, Shared &sh, uint16_t *ids) {
    const int tid = threadIdx.x, lane = tid & 31;
    for (int e = tid; e < p.E; e += kThreads) sh.count[e] = 0;
    __syncthreads();
    for (int i = tid; i < p.T * p.top; i += kThreads) {
        const int e = __ldcg(p.ids + i);  // from L2: another grid may have just written them
        const bool on = e >= 0 && e < p.E;
        ids[i] = on ? (uint16_t)e : kNone;
        if (on) atomicAdd(&sh.count[e], 1);
    }
    __syncthreads();
    if (tid < 32) {
        int busy = 0, cost = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int n = e0 + lane < p.E ? sh.count[e0 + lane] : 0;
            const uint32_t m = __ballot_sync(0xFFFFFFFFu, n > 0);
            int c = n > 0 ? tile_cost<C>(n) : 0, sum = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o) sum += v;
            }
            if (n > 0) {
                const int at = busy + __popc(m & ((1u << lane) - 1u));
                sh.act[at] = (uint16_t)(e0 + lane);
                sh.before[at] = cost + sum - c;
            }
            busy += __popc(m);
            cost += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        if (lane == 0) {
            sh.busy = busy;
            sh.cost = cost;
        }
    }
    __syncthreads();
}

// The same for at most 32 entries, in registers of every warp (an entry a
// lane) and without a barrier: the lanes that share the lane's expert, and,
// in the lowest of those, the cost before it; returned is the whole cost.
template <int C>
__device__ __forceinline__ int plan_few(const MoeParams &p, int &e, uint32_t &same, int &before) {
    const int lane = threadIdx.x & 31, n = p.T * p.top;
    e = lane < n ? __ldcg(p.ids + lane) : -1;
    if (e >= p.E) e = -1;
    same = __match_any_sync(0xFFFFFFFFu, e);
    const bool first = e >= 0 && (same & ((1u << lane) - 1u)) == 0;
    const int cost = first ? tile_cost<C>(__popc(same)) : 0;
    int sum = 0;
    before = 0;
    for (int i = 0; i < n; ++i) {
        const int ei = __shfl_sync(0xFFFFFFFFu, e, i), ci = __shfl_sync(0xFFFFFFFFu, cost, i);
        sum += ci;
        before += ei < e ? ci : 0;
    }
    if (!first) before = -1;
    return sum;
}

// Entries first .. first + MOST - 1 of expert e, in order.
template <int MOST>
__device__ __forceinline__ void list_entries(const MoeParams &p, int e, int first, Shared &sh,
                                             const uint16_t *ids) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int before = -first;
    for (int i0 = 0; i0 < p.T * p.top && before < MOST; i0 += kThreads) {
        const int i = i0 + tid;
        const bool on = i < p.T * p.top && ids[i] == e;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, on);
        if (lane == 0) sh.warp_sum[warp] = __popc(m);
        __syncthreads();
        int at = before + __popc(m & ((1u << lane) - 1u));
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += sh.warp_sum[w];
            before += sh.warp_sum[w];
        }
        if (on && at >= 0 && at < MOST) sh.list[at] = (uint16_t)i;
        __syncthreads();
    }
}

// Copies 16 (or 8) bytes of codes where `on`, without a branch: the lanes that
// have nothing to copy stay with the others.
template <int P>
__device__ __forceinline__ void copy_codes(uint32_t to, const uint8_t *from, bool on) {
    static_assert(P == 16 || P == 8, "16 or 8 bytes");
    if constexpr (P == 16)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t"
                     "@p cp.async.cg.shared.global.L2::128B [%0], [%1], 16;\n\t}" ::"r"(to),
                     "l"(from), "r"((uint32_t)on)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t"
                     "@p cp.async.ca.shared.global.L2::128B [%0], [%1], 8;\n\t}" ::"r"(to),
                     "l"(from), "r"((uint32_t)on)
                     : "memory");
}
// Copies P bytes of scales, or writes P bytes of zeros (and reads nothing).
template <int P>
__device__ __forceinline__ void copy_scales(uint32_t to, const uint8_t *from, bool on) {
    if constexpr (P == 16) {
        asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
                     "r"(on ? 16u : 0u)
                     : "memory");
    } else if constexpr (P == 8 || P == 4) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(P),
                     "r"(on ? (uint32_t)P : 0u)
                     : "memory");
    } else {
        uint16_t v = 0;
        if (on) asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(from) : "memory");
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(v) : "memory");
    }
}

// Where a chunk of `units` 64-value units of ncols columns lies: the columns,
// fp16 in MMA order (64 bytes of pitch: two rows' 16-byte reads differ in
// banks), then their group sums, two fp16 parts, whole blocks of scales. An
// odd number of 16 bytes as the sums' pitch puts 8 columns on all banks.
struct Layout {
    int pitch, sums, sum_lo, sum_pitch;
};
template <int UU, int BU>
__host__ __device__ constexpr Layout layout(int ncols, int units) {
    Layout l = {};
    l.pitch = (units + UU - 1) / UU * UU * 128 + 64;  // whole steps: units past the end count as zeros
    l.sums = ncols * l.pitch;
    l.sum_lo = (units + BU - 1) / BU * 16;
    l.sum_pitch = 2 * l.sum_lo + 16;
    return l;
}
template <int UU, int BU>
__host__ __device__ constexpr int layout_bytes(int ncols, int units) {
    return layout<UU, BU>(ncols, units).sums + ncols * layout<UU, BU>(ncols, units).sum_pitch;
}

// The listed columns for units u0 .. u0 + n - 1 as fp16 in MMA order, with
// their group sums times 2^-8 as two fp16 parts (22 bits).
template <int BITS, bool G32, bool PAIRS>
__device__ __forceinline__ void stage_columns(const MoeParams &p, int ncols, Shared &sh, int u0,
                                              int n, int padded, uint8_t *act, const Layout &l) {
    using Ord = Order<BITS, G32>;
    constexpr int SETS = G32 ? 2 : 1, KEPT = 2;  // quarters a thread has in flight
    const int tid = threadIdx.x, lane = tid & 31, U = p.K / 64;
    const bool wide = p.group == 128;
    const uint32_t quad = 0xFu << (lane & ~3);  // a unit's four lanes come together
    // a unit's quarter (column c, quarter k of K): 16 values in two pieces
    auto source = [&](int c, int k, size_t &second) {
        const int entry = sh.list[c];
        second = G32 ? 32 : 8;
        return (size_t)(PAIRS ? entry / p.top : entry) * p.K +
               (G32 ? (size_t)(k >> 2) * 64 + (k & 3) * 8 : (size_t)k * 16);
    };
    uint32_t raw[KEPT][PAIRS ? 8 : 16];
    auto load = [&](int c, int k, uint32_t(&w)[PAIRS ? 8 : 16]) {
        size_t second;
        const size_t at = source(c, k, second);
        source8<PAIRS>(p, at, w);
        source8<PAIRS>(p, at + second, w + (PAIRS ? 4 : 8));
    };
    const int peak_items = ncols * U * 4;
    const bool kept = u0 == 0 && n == U && n == padded && peak_items <= KEPT * kThreads;
    if (u0 == 0) {  // the columns' largest magnitudes
        if (tid < 32) sh.peak[tid] = 0u;
        __syncthreads();
        for (int i0 = tid; i0 < peak_items; i0 += KEPT * kThreads) {
#pragma unroll
            for (int r = 0; r < KEPT; ++r) {
                const int i = i0 + r * kThreads, c = i / (U * 4);
                if (i < peak_items) load(c, i - c * U * 4, raw[r]);
            }
#pragma unroll
            for (int r = 0; r < KEPT; ++r) {
                const int i = i0 + r * kThreads, c = i / (U * 4);
                if (i < peak_items) {
                    float v[16], m = 0.f;
                    widen16<PAIRS>(p, raw[r], v);
#pragma unroll
                    for (int k = 0; k < 16; ++k) m = fmaxf(m, fabsf(v[k]));
                    m = fmaxf(m, __shfl_xor_sync(quad, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(quad, m, 2));
                    if ((i & 3) == 0) atomicMax(&sh.peak[c], __float_as_uint(m));
                }
            }
        }
        __syncthreads();
    }
    const int items = ncols * padded * 4;
    for (int i0 = tid; i0 < items; i0 += KEPT * kThreads) {
        if (!kept) {
#pragma unroll
            for (int r = 0; r < KEPT; ++r) {
                const int i = i0 + r * kThreads, c = i / (padded * 4), k = i - c * padded * 4;
                if (i < items && (k >> 2) < n) load(c, u0 * 4 + k, raw[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < KEPT; ++r) {
            const int i = i0 + r * kThreads, c = i / (padded * 4), k = i - c * padded * 4;
            if (i >= items) continue;
            const int uu = k >> 2, qq = k & 3;
            uint4 *dst = reinterpret_cast<uint4 *>(act + (size_t)c * l.pitch + uu * 128) + qq;
            if (uu >= n) {  // past the end
                dst[0] = dst[4] = make_uint4(0u, 0u, 0u, 0u);
                continue;
            }
            float v[16];
            widen16<PAIRS>(p, raw[r], v);
            // 2^up puts the largest magnitude into [2^14, 2^15) (one below 2^-112
            // less high: 2^-126 is the smallest inverse that is a normal float)
            const int ex = (int)(sh.peak[c] >> 23);
            int up = ex == 255 ? 0 : 14 + 127 - ex;
            up = up > 126 ? 126 : up;
            const float f = __int_as_float((127 + up) << 23);
            if (k == 0) sh.undo[c] = __int_as_float((127 - up) << 23);
            float s = 0.f, s2 = 0.f;
#pragma unroll
            for (int m = 0; m < 16; ++m) v[m] *= f;
            // (the sums are of the values as the codes' products see them, so that
            // what rounds off of a value is multiplied by its weight, not by its
            // code's part of it)
            uint32_t o[8];
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                const float back = (float)(1 << Ord::pre(m)), down = 1.f / back;
                o[m] = pack_half2(v[Ord::lo(m)] * down, v[Ord::hi(m)] * down);
                const __half2 h = *reinterpret_cast<const __half2 *>(&o[m]);
                const float both = (__low2float(h) + __high2float(h)) * back;
                if (G32 && m >= 4)
                    s2 += both;
                else
                    s += both;
            }
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[4] = make_uint4(o[4], o[5], o[6], o[7]);
            s += __shfl_xor_sync(quad, s, 1);
            s += __shfl_xor_sync(quad, s, 2);
            if (G32) {
                s2 += __shfl_xor_sync(quad, s2, 1);
                s2 += __shfl_xor_sync(quad, s2, 2);
            }
            int at = G32 ? uu * 2 + qq : uu;  // its group's place
            if (!G32 && wide) {               // the other unit of the group: n is even, as is the lane's part
                s += __shfl_xor_sync(0xFFu << (lane & ~7), s, 4);
                at = (uu >> 3) * 8 + ((uu & 7) >> 1);
            }
            if (qq < SETS && !(wide && (uu & 1))) {
                const float v = (qq ? s2 : s) * 0.00390625f;
                const __half hi = __float2half_rn(v);
                __half *to = reinterpret_cast<__half *>(act + l.sums + (size_t)c * l.sum_pitch) + at;
                to[0] = hi;
                to[l.sum_lo / 2] = __float2half_rn(v - __half2float(hi));
            }
        }
    }
    // zeros in what is left of the blocks
    const int all = l.sum_lo / 2;
    if (wide || n * SETS < all)
        for (int i = tid; i < ncols * all; i += kThreads) {
            const int c = i / all, k = i - c * all;
            if (wide ? (k & 7) >= 4 || (k >> 3) * 8 + (k & 7) * 2 >= n : k >= n * SETS) {
                __half *to = reinterpret_cast<__half *>(act + l.sums + (size_t)c * l.sum_pitch) + k;
                to[0] = to[all] = __half(0.f);
            }
        }
}

// The same from packed rows: plain copies, asynchronous but for what is zero.
template <bool G32, bool PAIRS>
__device__ __forceinline__ void copy_columns(const MoeParams &p, int ncols, Shared &sh, int u0, int n, int padded,
                                             uint8_t *act, const Layout &l) {
    constexpr int BU = G32 ? 4 : 8;
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0);
    const MoePack m = moe_pack(PAIRS ? p.T : (int64_t)p.T * p.top, p.K, p.group);
    const int sums = (n + BU - 1) / BU;  // pieces of either part
    // a column a warp, or its halves, quarters or eighths where there are fewer
    const int parts = ncols > 4 ? 1 : ncols > 2 ? 2 : ncols == 2 ? 4 : 8, part = warp % parts;
    for (int c = warp / parts; c < ncols; c += kWarps / parts) {
        const int64_t row = PAIRS ? sh.list[c] / p.top : sh.list[c];
        const uint8_t *from = p.packed + row * p.K * 2 + (int64_t)u0 * 128;
        const uint32_t to = smem_u32(act) + (uint32_t)(c * l.pitch);
        for (int k = part * 32 + lane; k < n * 8; k += parts * 32) copy_codes<16>(to + k * 16, from + k * 16, true);
        if (part == 0) {
            const uint8_t *sum = p.packed + m.sums + row * m.blocks * 32 + u0 / BU * 16;
            const uint32_t to_sum = smem_u32(act) + (uint32_t)(l.sums + c * l.sum_pitch);
            for (int k = lane; k < sums; k += 32) {
                copy_codes<16>(to_sum + k * 16, sum + k * 16, true);
                copy_codes<16>(to_sum + l.sum_lo + k * 16, sum + m.blocks * 16 + k * 16, true);
            }
            if (lane < (padded - n) * 8)
                reinterpret_cast<uint4 *>(act + (size_t)c * l.pitch)[n * 8 + lane] = make_uint4(0u, 0u, 0u, 0u);
            if (lane == 0) sh.undo[c] = __ldcg(reinterpret_cast<const float *>(p.packed + m.undo) + row);
        }
    }
    cp_async_commit();
    cp_async_wait<0>();
}

// The sizes of a kernel for 8 NB columns, CTAS an SM.
template <int BITS, bool G32, bool PAIRS, int NB_, int CTAS_, bool PACKED_>
struct Kernel {
    static constexpr int NB = NB_, C = 8 * NB, UU = kUnits<BITS>, NW = kWords<BITS, G32>;
    static constexpr int SETS = G32 ? 2 : 1;     // groups of a unit whose sums are kept apart
    static constexpr int BU = G32 ? 4 : 8;       // units of a block of scales: 8 groups, 4 of 128
    static constexpr int ROWS = PAIRS ? 8 : 16;  // rows of a matrix in a tile
    static constexpr int UNIT = 8 * BITS;        // bytes of a unit's row
    static constexpr int CELL = 16 * UNIT, STAGE = UU * CELL;
    // Three steps in flight (two of 5 bits), and a block of scales for each, since
    // a step may be a tile's only one: with 24 warps an SM 72 KB of 4-bit codes.
    // Four and more measured slower (8 large experts: 205 us with three, 234
    // with four), and so did steps of twice the bytes.
    static constexpr int STAGES = STAGE <= 1024 ? 3 : 2, BLOCK = 512;  // 16 scales and biases of 8 groups
    static constexpr int CTAS = CTAS_, DYNAMIC = dynamic_bytes(CTAS);
    static constexpr int COLUMNS = layout_bytes<UU, BU>(C, 8) + 2 * kMaxEntries;
    static constexpr int RING = STAGES * (STAGE + BLOCK);  // a warp's
    static constexpr bool PACKED = PACKED_;        // columns from packed rows
    static constexpr bool SPLIT = BITS % 2 == 0;   // units apart in shared memory, else rows whole
    static constexpr int ROOM = DYNAMIC - kWarps * RING;  // for columns, less the entries' experts
    // 8 units of all columns fit beside the most entries, and the partial
    // sums of shared tiles where the rings were
    static_assert(COLUMNS <= ROOM && NB * 512 <= RING, "room");
};

// Tiles from .. to - 1 of expert e for the ncols listed entries.  The tiles go
// round the warps; those of the last, unfull round are shared by 2, 4 or 8
// warps, which split K.  Each warp has its codes and scales copied to shared
// memory a few steps ahead, from one tile to the next without a stop; the warps
// meet only where columns are staged.
template <class S, int BITS, bool G32, bool PAIRS>
__device__ __forceinline__ void run_tiles(const MoeParams &p, int e, int from, int to, int ncols, Shared &sh,
                                          uint8_t *dyn, int room, bool wait) {
    constexpr int NB = S::NB, UU = S::UU, BU = S::BU, SETS = S::SETS, STAGES = S::STAGES;
    const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, q = lane & 3;
    // (the shuffle tells the compiler that a warp's lanes agree on it)
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const int U = p.K / 64, groups = p.K / p.group;
    const bool wide = p.group == 128;

    // all of K's columns at once, or as many units of them as fit, a multiple of 8
    int cu = U;
    if (layout_bytes<UU, BU>(ncols, U) > room) {
        cu = (room - ncols * 128) / (ncols * (128 + 4 * SETS)) & ~7;
        cu = cu < 8 ? 8 : cu;
    }
    const Layout l = layout<UU, BU>(ncols, cu);
    uint8_t *act = dyn + kWarps * S::RING;
    const uint32_t ring = smem_u32(dyn + warp * S::RING), blocks = ring + STAGES * S::STAGE;
    float4 *slots = reinterpret_cast<float4 *>(dyn);

    const int full = (to - from) / kWarps, rest = to - from - full * kWarps;
    const int share = rest >= 5 ? 1 : rest >= 3 ? 2 : rest == 2 ? 4 : 8;
    const int rounds = full + (rest > 0);

    // what a lane copies of a tile's step: pieces of 16 bytes, PER a row (of 8
    // bytes where an odd width's rows are not multiples of 16: fine)
    constexpr int UNIT = S::UNIT, CELL = S::CELL, PER = UU * UNIT / 16, PIECES = (16 * PER + 31) / 32;
    const int64_t row_bytes = (int64_t)p.K * BITS / 8;
    const int64_t to_b = PAIRS ? reinterpret_cast<const uint8_t *>(p.w1) - reinterpret_cast<const uint8_t *>(p.w0)
                               : 8 * row_bytes;
    const int64_t to_t = S::ROWS * row_bytes;
    const bool fine = !S::SPLIT && (row_bytes & 8);
    auto piece_at = [&](int i) { return (lane + 32 * i) % PER * 16; };  // byte of the row's step
    auto piece_to = [&](int row, int at) {
        return (uint32_t)(S::SPLIT ? at / UNIT * CELL + row * UNIT + at % UNIT : row * UU * UNIT + at);
    };
    int64_t code_from[PIECES];
    uint32_t code_to[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int row = (lane + 32 * i) / PER;
        code_from[i] = (row & 7) * row_bytes + (row >= 8 ? to_b : 0) + piece_at(i);
        code_to[i] = piece_to(row, piece_at(i));
    }
    // and of a tile's block of scales: a row's scales or biases (16 rows of 16
    // bytes each), whole where rows allow, else in smaller pieces
    const int block_bytes = wide ? 8 : 16;
    const uint32_t even = (uint32_t)(reinterpret_cast<uintptr_t>(p.s0) | reinterpret_cast<uintptr_t>(p.b0) |
                                     reinterpret_cast<uintptr_t>(p.s1) | reinterpret_cast<uintptr_t>(p.b1)) |
                          (uint32_t)(groups * 2) | (uint32_t)block_bytes;
    const uint8_t *scale_row;  // the lane's row of the expert's first tile of the run
    {
        const int r = lane & 15;
        const bool second = PAIRS && r >= 8;
        const void *m = lane < 16 ? (second ? p.s1 : p.s0) : (second ? p.b1 : p.b0);
        scale_row = static_cast<const uint8_t *>(m) +
                    (((int64_t)e * p.R + (int64_t)from * S::ROWS + (PAIRS ? r & 7 : r)) * groups) * 2;
    }
    const uint8_t *w0 = reinterpret_cast<const uint8_t *>(p.w0) +
                        ((int64_t)e * p.R + (int64_t)from * S::ROWS) * row_bytes;
    const uint32_t shift = (uint32_t)first_bit<BITS, G32>(q) & 31u;
    const uint32_t mine = (uint32_t)(g * (S::SPLIT ? UNIT : UU * UNIT) + first_bit<BITS, G32>(q) / 32 * 4);

    float acc[NB][4];
    auto clear = [&]() {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nb][i] = 0.f;
    };
    // acc is in 2^-24 of the column's units
    auto write = [&](int tile, int c, float a, float b) {
        const float f = sh.undo[c];
        a = a * 16777216.f * f;
        b = b * 16777216.f * f;
        float *o = p.dst + (size_t)sh.list[c] * p.R + tile * S::ROWS + g;
        if constexpr (PAIRS) {
            // (exp(-a) passes the largest float at -88.7, where a exp(a) is still a
            // normal one; exp(a) alone is not, so b takes half of it)
            const float half = expf(0.5f * a);
            *o = a < -80.f ? a * half * (b * half) : a / (1.f + expf(-a)) * b;
        } else {
            o[0] = a;
            o[8] = b;
        }
    };
    // The warp's tile in a round and its steps of a chunk with nq steps.
    auto place = [&](int round, int nq, int &tile, int &beg, int &end) {
        if (round < full) {
            tile = round * kWarps + warp;
            beg = 0;
            end = nq;
        } else {
            const int i = warp / share, part = warp - i * share;
            tile = full * kWarps + i;
            beg = nq * part / share;
            end = i < rest ? nq * (part + 1) / share : beg;
        }
    };

    // Units u0 .. u0 + n - 1 of K for rounds r0 .. r1 - 1.
    auto stream = [&](int r0, int r1, int u0, int n) {
        const int nq = (n + UU - 1) / UU;
        // the step to fetch next
        int fround = r0, ftile, fk, fend, fu, fblock = 0;
        const uint8_t *src = nullptr;
        bool fresh = true;  // the first step of a tile
        uint32_t fr = ring;
        auto enter = [&]() {
            place(fround, nq, ftile, fk, fend);
            while (fk >= fend && ++fround < r1) place(fround, nq, ftile, fk, fend);
            fu = fk * UU;
            src = w0 + ftile * to_t + (int64_t)(u0 + fu) * UNIT;
            fresh = true;
        };
        enter();
        auto fetch = [&]() {
            if (fround < r1) {
                const int left = (n - fu) * UNIT;  // bytes of the row up to the chunk's end
                if (S::SPLIT || !fine) {
#pragma unroll
                    for (int i = 0; i < PIECES; ++i)
                        copy_codes<16>(fr + code_to[i], src + code_from[i],
                                       (16 * PER % 32 == 0 || lane + 32 * i < 16 * PER) &&
                                           (UU == 1 || piece_at(i) < left));
                } else {
                    for (int k = lane; k < 32 * PER; k += 32) {
                        const int row = k / (2 * PER), at = k % (2 * PER) * 8;
                        copy_codes<8>(fr + piece_to(row, at),
                                      src + (row & 7) * row_bytes + (row >= 8 ? to_b : 0) + at, at < left);
                    }
                }
                if (fresh || (fu & (BU - 1)) == 0) {
                    // the block of scales that this step lies in
                    const int b0 = (u0 + fu) / BU * block_bytes;  // of the row's bytes
                    const uint8_t *s = scale_row + (int64_t)ftile * (S::ROWS * 2) * groups + b0;
                    const uint32_t to_s = blocks + (uint32_t)(fblock * S::BLOCK + lane * 16);
                    const int have = groups * 2 - b0;  // bytes of the row from here on
                    if ((even & 15) == 0) {
                        copy_scales<16>(to_s, s, true);
                    } else if ((even & 7) == 0) {
                        copy_scales<8>(to_s, s, true);
                        copy_scales<8>(to_s + 8, s + 8, !wide && have >= 16);
                    } else if ((even & 3) == 0) {
#pragma unroll
                        for (int k = 0; k < 16; k += 4)
                            copy_scales<4>(to_s + k, s + k, k < block_bytes && have >= k + 4);
                    } else {
                        for (int k = 0; k < 16; k += 2)
                            copy_scales<2>(to_s + k, s + k, k < block_bytes && have >= k + 2);
                    }
                    fblock = fblock + 1 == STAGES ? 0 : fblock + 1;
                    fresh = false;
                }
                fu += UU;
                src += UU * UNIT;
                fr = fr + S::STAGE == ring + STAGES * S::STAGE ? ring : fr + S::STAGE;
                if (++fk >= fend && ++fround < r1) enter();
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < STAGES; ++i) fetch();

        if (wait) grid_dependency_wait();
        wait = false;
        __syncthreads();  // the last columns' readers are done
        if constexpr (S::PACKED)
            copy_columns<G32, PAIRS>(p, ncols, sh, u0, n, nq * UU, act, l);
        else
            stage_columns<BITS, G32, PAIRS>(p, ncols, sh, u0, n, nq * UU, act, l);
        __syncthreads();

        uint32_t xs[NB], ss[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int c = nb * 8 + g < ncols ? nb * 8 + g : 0;
            xs[nb] = smem_u32(act) + (uint32_t)(c * l.pitch + q * 16);
            ss[nb] = smem_u32(act) + (uint32_t)(l.sums + c * l.sum_pitch + 4 * q);
        }
        uint32_t rd = ring + mine;
        int block = -1;
        for (int round = r0; round < r1; ++round) {
            int tile, beg, end;
            place(round, nq, tile, beg, end);
            uint32_t sc = 0;
            for (int k = beg, u = beg * UU; k < end; ++k, u += UU) {
                cp_async_wait<STAGES - 1>();
                __syncwarp();
                if (k == beg || (u & (BU - 1)) == 0) {
                    block = block + 1 == STAGES ? 0 : block + 1;
                    sc = blocks + (uint32_t)(block * S::BLOCK);
                    if ((u & (BU - 1)) == 0) {
                        // the block's biases times the columns' group sums: acc is in
                        // 2^-24, these products in 2^-8
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            if (NB > 1 && nb * 8 >= ncols) continue;
                            uint32_t hi, lo;
                            lds<1>(ss[nb] + (uint32_t)(u / BU * 16), &hi);
                            lds<1>(ss[nb] + (uint32_t)(l.sum_lo + u / BU * 16), &lo);
                            uint32_t a0, a1;
                            lds<1>(sc + (uint32_t)(256 + g * 16 + 4 * q), &a0);
                            lds<1>(sc + (uint32_t)(384 + g * 16 + 4 * q), &a1);
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
                            mma_k8(d, a0, a1, hi);
                            mma_k8(d, a0, a1, lo);
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[nb][i] = fmaf(d[i], 1.52587890625e-05f, acc[nb][i]);
                        }
                    }
                }
                // scales of the step's groups, rows g and g + 8: the words that hold
                // them, and which half is unit 0's (with one group a step also unit 1's)
                constexpr int W = UU * SETS == 4 ? 2 : 1;
                const int at = wide ? (u & 7) >> 1 : (u & (BU - 1)) * SETS;
                const uint32_t pick = UU * SETS > 1 && !wide ? 0x3210u : at & 1 ? 0x3232u : 0x1010u;
                uint32_t sv[2][W];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    lds<W>(sc + (uint32_t)(b * 128 + g * 16 + (at & ~1) * 2), sv[b]);
                    if (UU * SETS < 4) sv[b][0] = prmt(sv[b][0], 0u, pick);
                }
#pragma unroll
                for (int i = 0; i < UU; ++i) {
                    uint32_t ra[8], rb[8];
                    {
                        uint32_t w[S::NW];
                        const uint32_t a = rd + (uint32_t)(S::SPLIT ? i * CELL : i * UNIT);
                        load_codes<BITS, G32>(a, w);
                        decode<BITS, G32>(w, shift, ra);
                        load_codes<BITS, G32>(a + 8 * (S::SPLIT ? UNIT : UU * UNIT), w);
                        decode<BITS, G32>(w, shift, rb);
                    }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        if (NB > 1 && nb * 8 >= ncols) continue;
                        const uint4 x = lds16(xs[nb] + (uint32_t)(u + i) * 128u);
                        const uint4 y = lds16(xs[nb] + (uint32_t)(u + i) * 128u + 64u);
                        float d[SETS][4];
                        mma0(d[0], ra[0], rb[0], ra[1], rb[1], x.x, x.y);
                        mma(d[0], ra[2], rb[2], ra[3], rb[3], x.z, x.w);
                        if constexpr (G32)
                            mma0(d[SETS - 1], ra[4], rb[4], ra[5], rb[5], y.x, y.y);
                        else
                            mma(d[0], ra[4], rb[4], ra[5], rb[5], y.x, y.y);
                        mma(d[SETS - 1], ra[6], rb[6], ra[7], rb[7], y.z, y.w);
#pragma unroll
                        for (int h = 0; h < SETS; ++h) {
                            const int z = i * SETS + h;
                            auto half = [&](int b) {
                                const __half2 v = *reinterpret_cast<const __half2 *>(&sv[b][z / 2]);
                                return z & 1 ? __high2float(v) : __low2float(v);
                            };
                            const float sa = half(0), sb = half(1);
                            acc[nb][0] = fmaf(sa, d[h][0], acc[nb][0]);
                            acc[nb][1] = fmaf(sa, d[h][1], acc[nb][1]);
                            acc[nb][2] = fmaf(sb, d[h][2], acc[nb][2]);
                            acc[nb][3] = fmaf(sb, d[h][3], acc[nb][3]);
                        }
                    }
                }
                __syncwarp();  // the stage is read: it may be filled again
                fetch();
                rd += S::STAGE;
                if (rd >= ring + STAGES * S::STAGE) rd -= STAGES * S::STAGE;
            }
            if (u0 + n >= U && (round < full || share == 1) && end > beg) {  // the tile is whole
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int c = nb * 8 + 2 * q + j;
                        if (c < ncols) write(from + tile, c, acc[nb][j], acc[nb][2 + j]);
                    }
                clear();
            }
        }
    };

    clear();
    for (int r0 = 0; r0 < rounds;) {
        const int r1 = cu == U ? rounds : r0 + 1;
        for (int u0 = 0; u0 < U; u0 += cu) stream(r0, r1, u0, U - u0 < cu ? U - u0 : cu);
        r0 = r1;
    }
    if (rest > 0 && share > 1) {
        // the warps' parts of the shared tiles, added in order
        __syncthreads();  // no copies are in flight, and the rings are read
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            slots[(warp * NB + nb) * 32 + lane] = make_float4(acc[nb][0], acc[nb][1], acc[nb][2], acc[nb][3]);
        __syncthreads();
        for (int i = warp; i < rest * NB; i += kWarps) {
            const int tile = i / NB, nb = i % NB;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = tile * share; w < (tile + 1) * share; ++w) {
                const float4 v = slots[(w * NB + nb) * 32 + lane];
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            }
            const int c = nb * 8 + 2 * q;
            if (c < ncols) write(from + full * kWarps + tile, c, s.x, s.z);
            if (c + 1 < ncols) write(from + full * kWarps + tile, c + 1, s.y, s.w);
        }
        __syncthreads();  // before the rings are filled again
    }
}

// A kernel takes columns 8 NB at a time; which one is launched is a matter of
// sizes alone (launch_sized below).
template <int BITS, bool G32, bool PAIRS, int NB, int CTAS, bool PACKED>
__global__ void __launch_bounds__(kThreads, Kernel<BITS, G32, PAIRS, NB, CTAS, PACKED>::CTAS) moe_kernel(const __grid_constant__ MoeParams p) {
    using S = Kernel<BITS, G32, PAIRS, NB, CTAS, PACKED>;
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ Shared sh;
    // The down grid reads ids and weights before it waits: this grid's
    // predecessor lets it start only once all that came before is complete.
    if (PAIRS) {
        grid_dependency_wait();
        launch_dependents();
    }
    // behind the rings: the columns, at the end the entries' experts
    const int room = S::ROOM - ((p.T * p.top * 2 + 15) & ~15);
    uint16_t *ids = reinterpret_cast<uint16_t *>(dyn + kWarps * S::RING + room);
    const bool few = p.T * p.top <= 32;
    int mine = -1, mine_before = -1;
    uint32_t same = 0u;
    int cost_all;
    if (few) {
        cost_all = plan_few<S::C>(p, mine, same, mine_before);
    } else {
        plan<S::C>(p, sh, ids);
        cost_all = sh.cost;
    }
    const int per = p.R / S::ROWS;  // tiles of an expert
    // this CTA takes the tiles that start at costs lo .. hi - 1 (at most 2^30)
    const int all = cost_all * per, G = (int)gridDim.x, each = all / G, rest = all - each * G;
    const int lo = each * (int)blockIdx.x + rest * (int)blockIdx.x / G;
    const int hi = each * ((int)blockIdx.x + 1) + rest * ((int)blockIdx.x + 1) / G;
    bool wait = !PAIRS;
    uint32_t mask = 0u;  // few: the lanes whose expert has tiles here
    int a = 0;           // else: the last busy expert that starts at or before lo
    if (few) {
        const int b = mine_before * per;
        mask = __ballot_sync(0xFFFFFFFFu, mine_before >= 0 && b < hi && b + tile_cost<S::C>(__popc(same)) * per > lo);
    } else {
        for (int step = AQ_MOE_MAX_EXPERTS / 2; step > 0; step >>= 1)
            if (a + step < sh.busy && sh.before[a + step] * per <= lo) a += step;
    }
    bool again = false;
    for (;;) {
        int e, count, start;
        uint32_t entries = 0u;
        if (few) {
            if (mask == 0u) break;
            const int i = __ffs(mask) - 1;
            mask &= mask - 1u;
            e = __shfl_sync(0xFFFFFFFFu, mine, i);
            entries = __shfl_sync(0xFFFFFFFFu, same, i);
            count = __popc(entries);
            start = __shfl_sync(0xFFFFFFFFu, mine_before, i) * per;
        } else {
            if (a >= sh.busy || sh.before[a] * per >= hi) break;
            e = sh.act[a];
            count = sh.count[e];
            start = sh.before[a++] * per;
        }
        const int cost = tile_cost<S::C>(count);
        const int from = lo > start ? (lo - start + cost - 1) / cost : 0;
        const int to = min((hi - start + cost - 1) / cost, per);
        if (from >= to) continue;
        for (int col0 = 0; col0 < count; col0 += S::C) {
            if (few) {
                if (again) __syncthreads();  // the last list's readers are done
                again = true;
                const int lane = threadIdx.x & 31, at = __popc(entries & ((1u << lane) - 1u)) - col0;
                if (threadIdx.x < 32 && (entries >> lane & 1u) && at >= 0 && at < S::C) sh.list[at] = (uint16_t)lane;
            } else {
                list_entries<S::C>(p, e, col0, sh, ids);
            }
            run_tiles<S, BITS, G32, PAIRS>(p, e, from, to, count - col0 < S::C ? count - col0 : S::C, sh, dyn,
                                           room, wait);
            wait = false;
        }
    }
    if (wait) grid_dependency_wait();
}

// The grid: every SM full, each CTA with an even run of tiles.
template <int BITS, bool G32, bool PAIRS, int NB, int CTAS, bool PACKED>
cudaError_t launch_one(const MoeParams &p, cudaStream_t stream) {
    using S = Kernel<BITS, G32, PAIRS, NB, CTAS, PACKED>;
    auto *kern = moe_kernel<BITS, G32, PAIRS, NB, CTAS, PACKED>;
    static std::atomic<uint64_t> ready{0};  // devices whose limit is raised, one bit each
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::DYNAMIC);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return moe_launch(kern, dim3((unsigned)(S::CTAS * num_sms())), kThreads, S::DYNAMIC, 1, stream, p);
}

// The kernel that moe_variant names, with its pack.
template <int BITS, bool G32, bool PAIRS>
cudaError_t launch_sized(const MoeParams &p, int variant, cudaStream_t stream) {
    switch (variant) {
        case MOE_8: return launch_one<BITS, G32, PAIRS, 1, 3, false>(p, stream);
        case MOE_8_PACKED: return launch_one<BITS, G32, PAIRS, 1, 3, true>(p, stream);
        case MOE_16: return launch_one<BITS, G32, PAIRS, 2, 2, true>(p, stream);
        default: return launch_one<BITS, G32, PAIRS, 4, 2, true>(p, stream);
    }
}

template <int BITS>
cudaError_t launch(const MoeParams &p, bool pairs, int variant, cudaStream_t stream) {
    if (p.group == 32)
        return pairs ? launch_sized<BITS, true, true>(p, variant, stream)
                     : launch_sized<BITS, true, false>(p, variant, stream);
    return pairs ? launch_sized<BITS, false, true>(p, variant, stream)
                 : launch_sized<BITS, false, false>(p, variant, stream);
}

// Packs a source row a CTA (moe_pack): what the products' CTAs would each do for
// the rows they need, done once.
constexpr int kPackUnits = 256;
template <int BITS, bool G32, bool PAIRS>
__global__ void __launch_bounds__(kThreads) pack_kernel(const __grid_constant__ MoeParams p, uint8_t *to) {
    constexpr int UU = kUnits<BITS>, BU = G32 ? 4 : 8;
    __shared__ Shared sh;
    extern __shared__ __align__(16) uint8_t act[];
    grid_dependency_wait();
    launch_dependents();
    const int tid = threadIdx.x, U = p.K / 64;
    const int64_t row = blockIdx.x;
    const MoePack m = moe_pack(PAIRS ? p.T : (int64_t)p.T * p.top, p.K, p.group);
    if (tid == 0) sh.list[0] = (uint16_t)(PAIRS ? row * p.top : row);
    __syncthreads();
    for (int u0 = 0; u0 < U; u0 += kPackUnits) {
        const int n = U - u0 < kPackUnits ? U - u0 : kPackUnits, sums = (n + BU - 1) / BU;
        const Layout l = layout<UU, BU>(1, n);
        stage_columns<BITS, G32, PAIRS>(p, 1, sh, u0, n, n, act, l);
        __syncthreads();
        uint4 *out = reinterpret_cast<uint4 *>(to + row * p.K * 2 + (int64_t)u0 * 128);
        for (int k = tid; k < n * 8; k += kThreads) out[k] = reinterpret_cast<const uint4 *>(act)[k];
        uint4 *sum = reinterpret_cast<uint4 *>(to + m.sums + row * m.blocks * 32) + u0 / BU;
        for (int k = tid; k < 2 * sums; k += kThreads) {
            const bool low = k >= sums;
            const int at = low ? k - sums : k;
            sum[(low ? m.blocks : 0) + at] = reinterpret_cast<const uint4 *>(act + l.sums + (low ? l.sum_lo : 0))[at];
        }
        __syncthreads();
    }
    if (tid == 0) reinterpret_cast<float *>(to + m.undo)[row] = sh.undo[0];
}

template <int BITS>
cudaError_t pack(const MoeParams &p, bool pairs, uint8_t *to, cudaStream_t stream) {
    void (*kern)(MoeParams, uint8_t *) =
        p.group == 32 ? (pairs ? pack_kernel<BITS, true, true> : pack_kernel<BITS, true, false>)
                      : (pairs ? pack_kernel<BITS, false, true> : pack_kernel<BITS, false, false>);
    const int units = p.K / 64 < kPackUnits ? p.K / 64 : kPackUnits;
    const int smem = p.group == 32 ? layout_bytes<kUnits<BITS>, 4>(1, units) : layout_bytes<kUnits<BITS>, 8>(1, units);
    return moe_launch(kern, dim3((unsigned)(pairs ? p.T : p.T * p.top)), kThreads, (size_t)smem, 1, stream, p, to);
}

}  // namespace moe_detail
}  // namespace aq
