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
//     even runs.  A CTA takes its run expert by expert, up to 16 tiles a pass.
//     Within a pass the (tile, 64-value unit) pairs, tile after tile, are
//     dealt to the 8 warps in even runs, so no shape leaves a warp idle; a
//     warp's part of tile t goes to slot t + warp (the pairs (tile, warp) that
//     occur lie on a monotone path, so their sums t + warp differ), and a
//     tile's slots are added in warp order: the result does not depend on
//     timing.
//   * Codes go from global memory to registers, several units ahead: lane
//     (g, q) of the MMA layout reads the 16 codes [16q, 16q + 16) of rows g and
//     g + 8.  The MMA's k order within a unit is whatever the decode gives
//     (Order<BITS>): the activations are staged in that order.
//   * A code masked in place in an fp16 with zero exponent is the exact
//     subnormal q * 2^(p - 24), p its bit position; the activation paired with
//     it carries 2^-p.  Activations are fp16 with one power of two per token
//     that puts the row's largest magnitude into [2^14, 2^15): bf16 and fp16
//     values above 2^-28 of it keep all their bits, smaller ones are off by
//     2^-39 of it at most; h (fp32) is rounded to fp16's 11 bits, 2^-11 of a
//     value at most, an eighth of what rounding it to bf16 would cost.
//     Sums of codes, group sums and everything after them are fp32.
//   * Tokens of an expert are MMA columns, 8, 16 or 32 at a time.
#pragma once

#include "aq_moe.h"
#include "aq_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <type_traits>

namespace aq {
namespace moe_detail {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxTiles = 16;        // tiles of a pass
constexpr int kRing = 6144;          // bytes of codes in flight a warp
constexpr int kDynamic = 109568;     // dynamic shared memory: two CTAs an SM
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
static_assert(2 * (kDynamic + sizeof(Shared) + 1024) <= 228 * 1024, "two CTAs an SM");

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

// A pass: tiles tile0 .. tile0 + nt - 1 of expert e for the ncols listed
// entries.  flat: the (tile, step) pairs are dealt to the warps in even runs;
// otherwise each warp, or `share` warps, keep TT tiles for the whole of K.
struct Pass {
    int e, tile0, nt, ncols;
};

// Shared memory behind the rings for a chunk of `units` 64-value units: the
// columns (fp16 in MMA order, 64 bytes of pitch so that two rows' 16-byte reads
// differ in banks), their group sums (two fp16 parts, a whole MMA step of 16
// groups), the tiles' scales and biases, and what sums need.  Pitches of an odd
// number of 16 bytes put 8 rows on all banks.
struct Layout {
    int pitch, sum_lo, sum_pitch, bias_at, scale_pitch;
    int sums, scales, total, slots, end;  // byte offsets
};
__host__ __device__ constexpr Layout layout(bool flat, int tt, int uu, int nb, int nt, int ncols, int group,
                                            int units) {
    Layout l = {};
    const int padded = (units + uu - 1) / uu * uu;  // whole steps: units past the end count as zeros
    const int have = group == 32 ? padded * 2 : group == 64 ? padded : (padded + 1) / 2;
    const int steps = (have + 15) / 16 * 32;  // bytes of whole MMA steps
    l.pitch = padded * 128 + 64;
    l.sum_lo = steps;
    l.sum_pitch = 2 * steps + 16;
    l.bias_at = (have * 2 + 15) / 16 * 16;
    l.scale_pitch = ((l.bias_at + steps) / 16 | 1) * 16;
    l.sums = ncols * l.pitch;
    l.scales = l.sums + ncols * l.sum_pitch;
    l.total = l.scales + nt * 16 * l.scale_pitch;
    l.slots = flat ? l.total + nt * nb * 512 : 0;
    l.end = flat ? l.slots + ((nt + tt - 1) / tt + kWarps - 1) * tt * nb * 512 : l.total;
    return l;
}
constexpr int kRoom = kDynamic - kWarps * kRing;  // less the entries' experts
// The most that 4 units take fits beside the most entries, and so do the slots
// of warps that keep their tiles.
static_assert(layout(false, 2, 2, 4, kMaxTiles, 32, 32, 4).end <= kRoom - 2 * kMaxEntries &&
              layout(true, 2, 2, 1, kMaxTiles, 8, 32, 4).end <= kRoom - 2 * kMaxEntries &&
              kWarps * 2 * 4 * 512 <= kRoom - 2 * kMaxEntries, "chunks");

// Units of a chunk: all, or the most that fit, steps of 16 where there are as
// many (the sums' MMA steps are whole then), else of 4.
__device__ __forceinline__ int chunk_units(bool flat, int tt, int uu, int nb, int nt, int ncols, int group,
                                           int U, int room) {
    if (layout(flat, tt, uu, nb, nt, ncols, group, U).end <= room) return U;
    int n = 4;
    while (n + 16 < U && layout(flat, tt, uu, nb, nt, ncols, group, n < 16 ? 16 : n + 16).end <= room)
        n = n < 16 ? 16 : n + 16;
    return n;
}

// Copies P bytes (a plain load and store for 2), asynchronously from 4 up.
template <int P>
__device__ __forceinline__ void copy_piece(uint32_t to, const uint8_t *from) {
    if constexpr (P == 16)
        asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else if constexpr (P == 8)
        asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
    else if constexpr (P == 4)
        asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
    else
        asm volatile("{\n\t.reg .b16 v;\n\tld.global.b16 v, [%1];\n\tst.shared.b16 [%0], v;\n\t}" ::"r"(to),
                     "l"(from)
                     : "memory");
}

// The scales and biases of the pass's rows for the groups of units u0 .. u0 +
// n - 1: each row's scales, at bias_at its biases, both with zeros up to the
// end of their room.
template <bool PAIRS, int P>
__device__ __forceinline__ void copy_scales(const MoeParams &p, const Pass &ps, int g0, int bytes, int groups,
                                            uint32_t scales, const Layout &l) {
    const int per = (bytes + P - 1) / P, rows = ps.nt * 16;
    // rows by threads, so that a row's pieces need no division; a wide row is
    // shared by several
    const int tid = threadIdx.x;
    int lanes = 1;
    while (lanes < 32 && lanes < per) lanes *= 2;
    for (int row = tid / lanes; row < rows; row += kThreads / lanes) {
        const int r = row & 15;
        const bool second = PAIRS && r >= 8;
        const int64_t at = (((int64_t)ps.e * p.R + (int64_t)(ps.tile0 + (row >> 4)) * (PAIRS ? 8 : 16) +
                             (PAIRS ? r & 7 : r)) * groups + g0) * 2;
        const uint8_t *s = static_cast<const uint8_t *>(second ? p.s1 : p.s0) + at;
        const uint8_t *b = static_cast<const uint8_t *>(second ? p.b1 : p.b0) + at;
        const uint32_t to = scales + (uint32_t)(row * l.scale_pitch);
        for (int k = tid % lanes; k < per; k += lanes) {
            copy_piece<P>(to + k * P, s + k * P);
            copy_piece<P>(to + l.bias_at + k * P, b + k * P);
        }
    }
}
template <bool PAIRS, int SETS>
__device__ __forceinline__ void stage_scales(const MoeParams &p, const Pass &ps, int u0, int n, int groups,
                                             uint32_t scales, const Layout &l) {
    const int wide = p.group == 128;
    const int g0 = wide ? u0 / 2 : u0 * SETS, ng = wide ? n / 2 : n * SETS;
    // the largest piece that the rows' starts and lengths allow
    const uint32_t all = (uint32_t)(reinterpret_cast<uintptr_t>(p.s0) | reinterpret_cast<uintptr_t>(p.b0) |
                                    reinterpret_cast<uintptr_t>(p.s1) | reinterpret_cast<uintptr_t>(p.b1)) |
                         (uint32_t)(groups * 2) | (uint32_t)(g0 * 2) | (uint32_t)(ng * 2);
    if ((all & 15) == 0)
        copy_scales<PAIRS, 16>(p, ps, g0, ng * 2, groups, scales, l);
    else if ((all & 7) == 0)
        copy_scales<PAIRS, 8>(p, ps, g0, ng * 2, groups, scales, l);
    else if ((all & 3) == 0)
        copy_scales<PAIRS, 4>(p, ps, g0, ng * 2, groups, scales, l);
    else
        copy_scales<PAIRS, 2>(p, ps, g0, ng * 2, groups, scales, l);
    auto zero = [&](int from, int to) {
        const int each = (to - from) / 2;
        for (int i = threadIdx.x; i < ps.nt * 16 * each; i += kThreads)
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(scales + (uint32_t)(i / each * l.scale_pitch + from + i % each * 2)),
                         "h"((short)0)
                         : "memory");
    };
    zero(2 * ng, l.bias_at);
    zero(l.bias_at + 2 * ng, l.bias_at + l.sum_lo);
}

// The pass's columns as fp16 in MMA order, with their group sums times 2^-8 as
// two fp16 parts (22 bits).
template <int BITS, bool G32, bool PAIRS>
__device__ __forceinline__ void stage_columns(const MoeParams &p, const Pass &ps, Shared &sh, int u0,
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
    const int peak_items = ps.ncols * U * 4;
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
    const int items = ps.ncols * padded * 4;
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
            // 2^up puts the largest magnitude into [2^14, 2^15)
            const int ex = (int)(sh.peak[c] >> 23);
            int up = ex == 0 || ex == 255 ? 0 : 14 + 127 - ex;
            up = up > 100 ? 100 : up;
            const float f = __int_as_float((127 + up) << 23);
            if (k == 0) sh.undo[c] = __int_as_float((127 - up) << 23);
            float s = 0.f, s2 = 0.f;
#pragma unroll
            for (int m = 0; m < 16; ++m) {
                v[m] *= f;
                const float h = __half2float(__float2half_rn(v[m]));
                if (G32 && m >= 8)
                    s2 += h;
                else
                    s += h;
            }
            uint32_t o[8];
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                const float down = 1.f / (float)(1 << Ord::pre(m));
                o[m] = pack_half2(v[Ord::lo(m)] * down, v[Ord::hi(m)] * down);
            }
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[4] = make_uint4(o[4], o[5], o[6], o[7]);
            s += __shfl_xor_sync(quad, s, 1);
            s += __shfl_xor_sync(quad, s, 2);
            if (G32) {
                s2 += __shfl_xor_sync(quad, s2, 1);
                s2 += __shfl_xor_sync(quad, s2, 2);
            }
            int at = G32 ? uu * 2 + qq : uu;  // its group
            if (!G32 && wide) {               // the other unit of the group: n is even, as is the lane's part
                s += __shfl_xor_sync(0xFFu << (lane & ~7), s, 4);
                at = uu >> 1;
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
    // zeros up to the last MMA step's end
    const int have = wide ? n / 2 : n * SETS, rest = l.sum_lo / 2 - have;
    for (int i = tid; i < ps.ncols * rest; i += kThreads) {
        __half *to = reinterpret_cast<__half *>(act + l.sums + (size_t)(i / rest) * l.sum_pitch) + have + i % rest;
        to[0] = to[l.sum_lo / 2] = __half(0.f);
    }
}

// TT tiles side by side share the activations that a step reads from shared
// memory; 8 NB columns.  (With an odd number of tiles the last one is taken
// twice and counted once.)  staged: the last pass left these columns, for all
// of K, in shared memory; returned is whether this one does.
template <int BITS, bool G32, bool PAIRS, bool FLAT, int TT, int NB>
__device__ __forceinline__ bool run_pass(const MoeParams &p, const Pass &ps, Shared &sh, uint8_t *dyn,
                                         int room, bool wait, bool staged) {
    constexpr int NW = kWords<BITS, G32>, UU = kUnits<BITS>;
    constexpr int SETS = G32 ? 2 : 1;      // groups of a unit whose sums are kept apart
    constexpr int ROWS = PAIRS ? 8 : 16;   // rows of a matrix in a tile
    constexpr int UNIT = 8 * BITS;         // bytes of a unit's row
    constexpr int CELL = 16 * UNIT, STAGE = TT * UU * CELL;
    constexpr int STAGES = kRing / STAGE < 8 ? kRing / STAGE : 8;
    constexpr bool SPLIT = BITS % 2 == 0;  // units apart in shared memory, else rows whole
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    const int U = p.K / 64, nt = ps.nt, ns = (nt + TT - 1) / TT;
    const int groups = p.K / p.group;
    const bool wide = p.group == 128;

    const int cu = chunk_units(FLAT, TT, UU, NB, nt, ps.ncols, p.group, U, room);
    const Layout l = layout(FLAT, TT, UU, NB, nt, ps.ncols, p.group, cu);
    const uint32_t ring = smem_u32(dyn + warp * kRing);
    uint8_t *act = dyn + kWarps * kRing;
    float4 *total = reinterpret_cast<float4 *>(act + l.total);
    float4 *slots = reinterpret_cast<float4 *>(act + l.slots);

    const int64_t row_bytes = (int64_t)p.K * BITS / 8;
    const int64_t to_b = PAIRS ? reinterpret_cast<const uint8_t *>(p.w1) - reinterpret_cast<const uint8_t *>(p.w0)
                               : 8 * row_bytes;
    const int64_t to_t = ROWS * row_bytes;
    const uint8_t *w0 = reinterpret_cast<const uint8_t *>(p.w0) +
                        ((int64_t)ps.e * p.R + (int64_t)ps.tile0 * ROWS) * row_bytes;
    // what a lane copies of a tile's step: pieces of 16 bytes, PER a row (of 8
    // bytes where an odd width's rows are not multiples of 16: fine)
    constexpr int PER = UU * UNIT / 16, PIECES = (16 * PER + 31) / 32;
    const bool fine = !SPLIT && (row_bytes & 8);
    auto piece_at = [&](int i) { return (lane + 32 * i) % PER * 16; };  // byte of the row's step
    auto piece_to = [&](int row, int at) {
        return (uint32_t)(SPLIT ? at / UNIT * CELL + row * UNIT + at % UNIT : row * UU * UNIT + at);
    };
    int64_t from[PIECES];
    uint32_t to[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int row = (lane + 32 * i) / PER;
        from[i] = (row & 7) * row_bytes + (row >= 8 ? to_b : 0) + piece_at(i);
        to[i] = piece_to(row, piece_at(i));
    }
    const uint32_t shift = (uint32_t)first_bit<BITS, G32>(q) & 31u;
    const uint32_t mine = (uint32_t)(g * (SPLIT ? UNIT : UU * UNIT) + first_bit<BITS, G32>(q) / 32 * 4);
    const int share = FLAT ? 1 : ns >= 5 ? 1 : ns >= 3 ? 2 : ns == 2 ? 4 : 8;

    float acc[TT][NB][4];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][nb][i] = 0.f;

    for (int u0 = 0; u0 < U; u0 += cu) {
        const int n = U - u0 < cu ? U - u0 : cu;     // units of this chunk
        const int nq = (n + UU - 1) / UU;            // steps of a tile
        int st, beg, end;                            // first tile (of TT), steps counted from it
        if (FLAT) {
            beg = ns * nq * warp / kWarps;
            end = ns * nq * (warp + 1) / kWarps;
            st = beg / nq;
            beg -= st * nq;
            end -= st * nq;
        } else {
            st = warp / share;
            beg = nq * (warp % share) / share;
            end = st < ns ? nq * (warp % share + 1) / share : beg;
        }

        // the step to fetch next: its tiles, its first unit
        int fs = st, fu = beg * UU, fk = beg;
        const uint8_t *src = w0 + (int64_t)(st * TT) * to_t + (int64_t)(u0 + fu) * UNIT;
        int64_t next = TT == 2 && st * 2 + 1 < nt ? to_t : 0;
        const int64_t wrap = TT * to_t - (int64_t)nq * UU * UNIT;
        uint32_t fr = ring;
        auto fetch = [&]() {
            if (fk < end) {
                const int left = (n - fu) * UNIT;  // bytes of the row up to the chunk's end
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const uint8_t *s = src + (t ? next : 0);
                    if (SPLIT || !fine) {
#pragma unroll
                        for (int i = 0; i < PIECES; ++i)
                            if ((16 * PER % 32 == 0 || lane + 32 * i < 16 * PER) && (UU == 1 || piece_at(i) < left))
                                copy_piece<16>(fr + t * UU * CELL + to[i], s + from[i]);
                    } else {
                        for (int k = lane; k < 32 * PER; k += 32) {
                            const int row = k / (2 * PER), at = k % (2 * PER) * 8;
                            if (at < left)
                                copy_piece<8>(fr + t * UU * CELL + piece_to(row, at),
                                              s + (row & 7) * row_bytes + (row >= 8 ? to_b : 0) + at);
                        }
                    }
                }
                fu += UU;
                src += UU * UNIT;
                if (fu >= n) {
                    fu = 0;
                    ++fs;
                    src += wrap;
                    if (TT == 2) next = fs * 2 + 1 < nt ? to_t : 0;
                }
                ++fk;
                fr = fr + STAGE == ring + STAGES * STAGE ? ring : fr + STAGE;
            }
            cp_async_commit();
        };
        __syncthreads();  // the last chunk's or pass's readers are done
        const uint32_t scale0 = smem_u32(act + l.scales);
        stage_scales<PAIRS, SETS>(p, ps, u0, n, groups, scale0, l);
        cp_async_commit();
#pragma unroll
        for (int i = 0; i < STAGES; ++i) fetch();
        if (wait && u0 == 0) grid_dependency_wait();
        if (!(FLAT && staged && cu == U))
            stage_columns<BITS, G32, PAIRS>(p, ps, sh, u0, n, nq * UU, act, l);
        cp_async_wait<STAGES>();  // the scales
        __syncthreads();

        uint32_t xs[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int c = nb * 8 + g;
            xs[nb] = smem_u32(act) + (uint32_t)((c < ps.ncols ? c : 0) * l.pitch + q * 16);
        }
        int u = beg * UU;
        uint32_t rd = ring + mine;
        // the scales of rows g and g + 8 of the warp's tiles
        const uint32_t sp = (uint32_t)l.scale_pitch;
        uint32_t sc0 = scale0 + (uint32_t)(st * TT * 16 + g) * sp;
        uint32_t sc1 = TT == 2 && st * 2 + 1 < nt ? 16u * sp : 0u;
        // The chunk's biases times group sums, 16 groups a product, by the warp
        // that takes a tile's last step: acc is in 2^-24, these products in 2^-8.
        auto add_biases = [&]() {
            const uint32_t bias = (uint32_t)(l.bias_at + 4 * q);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                if (NB > 1 && nb * 8 >= ps.ncols) continue;
                const int c = nb * 8 + g;
                const uint32_t sum = smem_u32(act) + (uint32_t)(l.sums + (c < ps.ncols ? c : 0) * l.sum_pitch + 4 * q);
                float d[TT][4];
#pragma unroll
                for (int t = 0; t < TT; ++t) d[t][0] = d[t][1] = d[t][2] = d[t][3] = 0.f;
                for (int k = 0; k < l.sum_lo; k += 32) {
                    uint32_t h0, h1, l0, l1;
                    lds<1>(sum + k, &h0);
                    lds<1>(sum + k + 16, &h1);
                    lds<1>(sum + l.sum_lo + k, &l0);
                    lds<1>(sum + l.sum_lo + k + 16, &l1);
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        const uint32_t o = sc0 + (t ? sc1 : 0u) + bias + k;
                        uint32_t a0, a1, a2, a3;
                        lds<1>(o, &a0);
                        lds<1>(o + 8u * sp, &a1);
                        lds<1>(o + 16u, &a2);
                        lds<1>(o + 8u * sp + 16u, &a3);
                        mma(d[t], a0, a1, a2, a3, h0, h1);
                        mma(d[t], a0, a1, a2, a3, l0, l1);
                    }
                }
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[t][nb][i] = fmaf(d[t][i], 1.52587890625e-05f, acc[t][nb][i]);
            }
        };
        for (int k = beg; k < end; ++k) {
            cp_async_wait<STAGES - 1>();
            __syncwarp();
            // scales of the step's groups, rows g and g + 8 of each tile: the words
            // that hold them, and which half is unit 0's (with one group a step
            // also unit 1's)
            constexpr int W = UU * SETS == 4 ? 2 : 1;
            const int at = wide ? u >> 1 : u * SETS;
            const uint32_t pick = UU * SETS > 1 && !wide ? 0x3210u : at & 1 ? 0x3232u : 0x1010u;
            uint32_t sc[TT][2][W];
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    lds<W>(sc0 + (t ? sc1 : 0u) + (b ? 8u * sp : 0u) + (uint32_t)(at & ~1) * 2u, sc[t][b]);
                    if (UU * SETS < 4) sc[t][b][0] = prmt(sc[t][b][0], 0u, pick);
                }
#pragma unroll
            for (int i = 0; i < UU; ++i) {
                uint32_t ra[TT][8], rb[TT][8];
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    uint32_t w[NW];
                    const uint32_t a = rd + (uint32_t)((t * UU + (SPLIT ? i : 0)) * CELL + (SPLIT ? 0 : i * UNIT));
                    load_codes<BITS, G32>(a, w);
                    decode<BITS, G32>(w, shift, ra[t]);
                    load_codes<BITS, G32>(a + 8 * (SPLIT ? UNIT : UU * UNIT), w);
                    decode<BITS, G32>(w, shift, rb[t]);
                }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    if (NB > 1 && nb * 8 >= ps.ncols) continue;
                    const uint4 x = lds16(xs[nb] + (uint32_t)(u + i) * 128u);
                    const uint4 y = lds16(xs[nb] + (uint32_t)(u + i) * 128u + 64u);
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        float d[SETS][4];
                        mma0(d[0], ra[t][0], rb[t][0], ra[t][1], rb[t][1], x.x, x.y);
                        mma(d[0], ra[t][2], rb[t][2], ra[t][3], rb[t][3], x.z, x.w);
                        if constexpr (G32)
                            mma0(d[SETS - 1], ra[t][4], rb[t][4], ra[t][5], rb[t][5], y.x, y.y);
                        else
                            mma(d[0], ra[t][4], rb[t][4], ra[t][5], rb[t][5], y.x, y.y);
                        mma(d[SETS - 1], ra[t][6], rb[t][6], ra[t][7], rb[t][7], y.z, y.w);
                        float(&o)[4] = acc[t][nb];
#pragma unroll
                        for (int h = 0; h < SETS; ++h) {
                            const int z = i * SETS + h;
                            auto half = [&](int b) {
                                const __half2 p2 = *reinterpret_cast<const __half2 *>(&sc[t][b][z / 2]);
                                return z & 1 ? __high2float(p2) : __low2float(p2);
                            };
                            const float sa = half(0), sb = half(1);
                            o[0] = fmaf(sa, d[h][0], o[0]);
                            o[1] = fmaf(sa, d[h][1], o[1]);
                            o[2] = fmaf(sb, d[h][2], o[2]);
                            o[3] = fmaf(sb, d[h][3], o[3]);
                        }
                    }
                }
            }
            __syncwarp();  // the stage is read: it may be filled again
            fetch();
            rd += STAGE;
            if (rd >= ring + STAGES * STAGE) rd -= STAGES * STAGE;
            u += UU;
            if (u >= n) add_biases();
            if (FLAT && (u >= n || k + 1 == end)) {
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        float(&o)[4] = acc[t][nb];
                        slots[(((st + warp) * TT + t) * NB + nb) * 32 + lane] =
                            make_float4(o[0], o[1], o[2], o[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[i] = 0.f;
                    }
                u = 0;
                ++st;
                sc0 += (uint32_t)(TT * 16) * sp;
                if (TT == 2) sc1 = st * 2 + 1 < nt ? 16u * sp : 0u;
            }
        }
        __syncthreads();
        const bool done = u0 + n >= U;
        if (!FLAT) {
            if (!done) continue;
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    slots[((warp * TT + t) * NB + nb) * 32 + lane] =
                        make_float4(acc[t][nb][0], acc[t][nb][1], acc[t][nb][2], acc[t][nb][3]);
            __syncthreads();
        }

        // the tiles' sums, in warp order; after the last chunk the results
        for (int i = tid; i < nt * NB * 32; i += kThreads) {
            const int tt = i / (NB * 32), s0 = tt / TT, nb = i / 32 % NB, ln = i & 31;
            float4 s = !FLAT || u0 == 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : total[i];
            const int first = FLAT ? 0 : s0 * share, last = FLAT ? kWarps : first + share;
            for (int w = first; w < last; ++w) {
                if (!FLAT || max(ns * nq * w / kWarps, s0 * nq) < min(ns * nq * (w + 1) / kWarps, (s0 + 1) * nq)) {
                    const float4 v = slots[(((FLAT ? s0 + w : w) * TT + tt % TT) * NB + nb) * 32 + ln];
                    s.x += v.x;
                    s.y += v.y;
                    s.z += v.z;
                    s.w += v.w;
                }
            }
            if (!done) {
                total[i] = s;
                continue;
            }
            const int row = (ps.tile0 + tt) * ROWS + (ln >> 2);
            const float part[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = nb * 8 + 2 * (ln & 3) + j;
                if (c >= ps.ncols) continue;
                const float a = part[j] * 16777216.f * sh.undo[c];
                const float b = part[2 + j] * 16777216.f * sh.undo[c];
                float *to = p.dst + (size_t)sh.list[c] * p.R + row;
                if constexpr (PAIRS) {
                    *to = a / (1.f + expf(-a)) * b;
                } else {
                    to[0] = a;
                    to[8] = b;
                }
            }
        }
    }
    return FLAT && cu == U;
}

// A kernel takes columns 8 NB at a time; which one is launched is a matter of
// sizes alone (variant below).
template <int BITS, bool G32, bool PAIRS, bool FLAT, int TT, int NB>
__global__ void __launch_bounds__(kThreads, 2) moe_kernel(const __grid_constant__ MoeParams p) {
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ Shared sh;
    // The down grid reads ids and weights before it waits: this grid's
    // predecessor lets it start only once all that came before is complete.
    if (PAIRS) {
        grid_dependency_wait();
        launch_dependents();
    }
    // behind the rings: room for the passes, at the end the entries' experts
    const int room = kRoom - ((p.T * p.top * 2 + 15) & ~15);
    uint16_t *ids = reinterpret_cast<uint16_t *>(dyn + kWarps * kRing + room);
    plan<8 * NB>(p, sh, ids);
    const int per = p.R / (PAIRS ? 8 : 16);  // tiles of an expert
    // this CTA takes the tiles that start at costs lo .. hi - 1 (at most 2^30)
    const int all = sh.cost * per, G = (int)gridDim.x, each = all / G, rest = all - each * G;
    const int lo = each * (int)blockIdx.x + rest * (int)blockIdx.x / G;
    const int hi = each * ((int)blockIdx.x + 1) + rest * ((int)blockIdx.x + 1) / G;
    bool wait = !PAIRS;
    int a = 0;  // the last busy expert that starts at or before lo
    for (int step = AQ_MOE_MAX_EXPERTS / 2; step > 0; step >>= 1)
        if (a + step < sh.busy && sh.before[a + step] * per <= lo) a += step;
    for (; a < sh.busy && sh.before[a] * per < hi; ++a) {
        const int e = sh.act[a], count = sh.count[e], cost = tile_cost<8 * NB>(count);
        const int start = sh.before[a] * per;
        const int from = lo > start ? (lo - start + cost - 1) / cost : 0;
        const int to = min((hi - start + cost - 1) / cost, per);
        if (from >= to) continue;
        for (int col0 = 0; col0 < count; col0 += 8 * NB) {
            list_entries<8 * NB>(p, e, col0, sh, ids);
            Pass ps;
            ps.e = e;
            ps.ncols = count - col0 < 8 * NB ? count - col0 : 8 * NB;
            bool staged = false;
            for (ps.tile0 = from; ps.tile0 < to; ps.tile0 += ps.nt) {
                ps.nt = to - ps.tile0 < kMaxTiles ? to - ps.tile0 : kMaxTiles;
                // fewer tiles where 16 leave no room for chunks of 16 units
                if (ps.nt > kMaxTiles / 2 &&
                    chunk_units(FLAT, TT, kUnits<BITS>, NB, ps.nt, ps.ncols, p.group, p.K / 64, room) <
                        (p.K < 1024 ? p.K / 64 : 16))
                    ps.nt = kMaxTiles / 2;
                staged = run_pass<BITS, G32, PAIRS, FLAT, TT, NB>(p, ps, sh, dyn, room, wait, staged);
                wait = false;
            }
        }
    }
    if (wait) grid_dependency_wait();
}

// The grid: two CTAs an SM, each with an even run of tiles.
template <int BITS, bool G32, bool PAIRS, bool FLAT, int TT, int NB>
cudaError_t launch_one(const MoeParams &p, cudaStream_t stream) {
    auto *kern = moe_kernel<BITS, G32, PAIRS, FLAT, TT, NB>;
    static std::atomic<uint64_t> ready{0};  // devices whose limit is raised, one bit each
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynamic);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return moe_launch(kern, dim3(2u * (unsigned)num_sms()), kThreads, kDynamic, 1, stream, p);
}

// Which kernel: by the tokens a busy expert has on average and the tiles a CTA
// gets, were all experts picked alike.
template <int BITS, bool G32, bool PAIRS>
cudaError_t launch_sized(const MoeParams &p, cudaStream_t stream) {
    const double picked = (double)p.T * p.top;
    const double busy = p.E * -std::expm1(p.T * std::log1p(-(double)(p.top < p.E ? p.top : p.E - 0.5) / p.E));
    const double tokens = picked / busy, tiles = busy * (p.R / (PAIRS ? 8 : 16)) / (2.0 * num_sms());
    if (p.T <= 8 || tokens <= 2.0) {
        if (tiles <= 3.0) return launch_one<BITS, G32, PAIRS, true, 1, 1>(p, stream);
        if (tiles <= 8.0) return launch_one<BITS, G32, PAIRS, true, 2, 1>(p, stream);
        return launch_one<BITS, G32, PAIRS, false, 2, 1>(p, stream);
    }
    if (p.T <= 16 || tokens <= 10.0) return launch_one<BITS, G32, PAIRS, false, 2, 2>(p, stream);
    return launch_one<BITS, G32, PAIRS, false, 2, 4>(p, stream);
}

template <int BITS>
cudaError_t launch(const MoeParams &p, bool pairs, cudaStream_t stream) {
    if (p.group == 32)
        return pairs ? launch_sized<BITS, true, true>(p, stream)
                     : launch_sized<BITS, true, false>(p, stream);
    return pairs ? launch_sized<BITS, false, true>(p, stream)
                 : launch_sized<BITS, false, false>(p, stream);
}

}  // namespace moe_detail
}  // namespace aq
