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

namespace aq {
namespace moe_detail {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxTiles = 16;      // tiles of a pass
constexpr int kDynamic = 90112;    // dynamic shared memory: two CTAs an SM
constexpr uint16_t kNone = 0xFFFF;
constexpr int kMaxEntries = AQ_MOE_MAX_TOKENS * AQ_MOE_MAX_TOP;

// How the 16 codes of a lane's segment land in the 8 registers of fp16 pairs:
// register p holds codes lo(p) and hi(p) at bit position pre(p).
template <int B>
struct Order {
    __host__ __device__ static constexpr int lo(int p) {
        return B == 4 ? (p / 4) * 8 + p % 4 : B == 8 ? (p / 2) * 4 + p % 2 : p;
    }
    __host__ __device__ static constexpr int hi(int p) {
        return B == 4 ? lo(p) + 4 : B == 8 ? lo(p) + 2 : p + 8;
    }
    __host__ __device__ static constexpr int pre(int p) {
        return B == 2   ? (p < 5 ? 2 * p : 2 * (p - 5))
               : B == 3 ? (p < 3 ? 3 * p : p < 5 ? 3 * (p - 3) : 3 * (p - 5))
               : B == 4 ? 4 * (p & 1)
               : B == 5 ? (p % 3 == 1 ? 5 : 0)
                        : 0;
    }
};

// 32-bit words that hold a lane's 16 codes of one row and unit (odd widths
// start in the middle of a word in odd lanes).
template <int B>
constexpr int kWords = B == 2 ? 1 : B == 3 || B == 4 ? 2 : B == 8 ? 4 : 3;
// Units in flight a lane: about 32 registers.
template <int B>
constexpr int kAhead = B == 8 ? 4 : kWords<B> == 3 ? 5 : 8;

template <int B>
__device__ __forceinline__ void load_codes(const uint32_t *p, uint32_t (&w)[kWords<B>]) {
    if constexpr (B == 4) {
        asm("ld.global.nc.L1::no_allocate.L2::128B.v2.u32 {%0, %1}, [%2];"
            : "=r"(w[0]), "=r"(w[1])
            : "l"(p));
    } else if constexpr (B == 8) {
        asm("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
            : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
            : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < kWords<B>; ++i)
            asm("ld.global.nc.L2::128B.u32 %0, [%1];" : "=r"(w[i]) : "l"(p + i));
    }
}

// A lane's 16 codes as 8 registers of two fp16 subnormals each; sh: 0, or 16
// where the codes start in the upper half of the first word.
template <int B>
__device__ __forceinline__ void decode(const uint32_t (&w)[kWords<B>], uint32_t sh,
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

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 source values, from x (fp16 or bf16) or h (fp32).
template <bool PAIRS>
__device__ __forceinline__ void source16(const MoeParams &p, size_t at, float (&v)[16]) {
    if constexpr (PAIRS) {
        const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.src) + at);
        const uint4 a = s[0], b = s[1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (p.dtype == AQ_BF16) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    } else {
        const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p.src) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 f = s[i];
            v[4 * i] = f.x;
            v[4 * i + 1] = f.y;
            v[4 * i + 2] = f.z;
            v[4 * i + 3] = f.w;
        }
    }
}

struct Shared {
    uint16_t act[AQ_MOE_MAX_EXPERTS];  // the busy experts, ascending
    uint16_t ids[kMaxEntries];         // every entry's expert, kNone without one
    uint16_t list[kMaxEntries];        // entries t * top + j of the current expert
    int count[AQ_MOE_MAX_EXPERTS];     // entries of each expert
    uint32_t peak[32];                 // a column's largest magnitude, as bits
    float undo[32];                    // a column's inverse power of two
    int warp_sum[kWarps];
    int busy, listed;
};

// Counts the entries of every expert and lists the busy experts in order.
__device__ __forceinline__ void plan(const MoeParams &p, Shared &sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < p.E; e += kThreads) sh.count[e] = 0;
    __syncthreads();
    for (int i = tid; i < p.T * p.top; i += kThreads) {
        const int e = __ldcg(p.ids + i);  // from L2: another grid may have just written them
        const bool on = e >= 0 && e < p.E;
        sh.ids[i] = on ? (uint16_t)e : kNone;
        if (on) atomicAdd(&sh.count[e], 1);
    }
    __syncthreads();
    int before = 0;
    for (int e0 = 0; e0 < p.E; e0 += kThreads) {
        const int e = e0 + tid;
        const bool on = e < p.E && sh.count[e] > 0;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, on);
        if (lane == 0) sh.warp_sum[warp] = __popc(m);
        __syncthreads();
        int at = before;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += sh.warp_sum[w];
            before += sh.warp_sum[w];
        }
        if (on) sh.act[at + __popc(m & ((1u << lane) - 1u))] = (uint16_t)e;
        __syncthreads();
    }
    if (tid == 0) sh.busy = before;
    __syncthreads();
}

// The entries of expert e, in order.
__device__ __forceinline__ void list_entries(const MoeParams &p, int e, Shared &sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int before = 0;
    for (int i0 = 0; i0 < p.T * p.top; i0 += kThreads) {
        const int i = i0 + tid;
        const bool on = i < p.T * p.top && sh.ids[i] == e;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, on);
        if (lane == 0) sh.warp_sum[warp] = __popc(m);
        __syncthreads();
        int at = before;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += sh.warp_sum[w];
            before += sh.warp_sum[w];
        }
        if (on) sh.list[at + __popc(m & ((1u << lane) - 1u))] = (uint16_t)i;
        __syncthreads();
    }
}

// 64-value units of K whose activations, group sums and scales fit in shared
// memory beside the slots and totals of nt tiles.
__host__ __device__ constexpr int units_that_fit(int nt, int ncols, int nb, int sets) {
    const int fixed = (2 * nt + kWarps - 1) * nb * 512 + 128 + nt * 16 * 8 + ncols * 64 + 64;
    const int each = 8 * nb * sets * 4 + nt * 16 * sets * 4 + ncols * 128;
    return (kDynamic - fixed) / each;
}
// With 32 columns and groups of 32 (the most a unit takes), four tiles still
// leave chunks of 8 units and more.
static_assert(units_that_fit(4, 32, 4, 2) >= 8 && units_that_fit(8, 16, 2, 2) >= 8, "chunks");

// A pass: tiles tile0 .. tile0 + nt - 1 of expert e for the ncols entries at
// list[col0].
struct Pass {
    int e, tile0, nt, col0, ncols;
};

template <int BITS, bool G32, bool PAIRS, int NB>
__device__ __forceinline__ void run_pass(const MoeParams &p, const Pass &ps, Shared &sh,
                                         uint8_t *dyn, bool wait) {
    constexpr int NW = kWords<BITS>, AHEAD = kAhead<BITS>, C = 8 * NB;
    constexpr int SETS = G32 ? 2 : 1;  // groups of a unit whose sums are kept apart
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    const int U = p.K / 64, nt = ps.nt;
    const int groups = p.K / p.group;

    // shared memory: slots, totals, group sums, zeros, (scale, bias) pairs, activations
    float4 *slots = reinterpret_cast<float4 *>(dyn);
    float4 *total = slots + (nt + kWarps - 1) * NB * 32;
    int cu = units_that_fit(nt, ps.ncols, NB, SETS);  // units of a chunk; even: whole groups of 128
    cu = cu >= U ? U : cu & ~1;
    const int ng_all = p.group == 128 ? (cu + 1) / 2 : cu * SETS;
    const int sp = ng_all | 1;  // pairs of a row: an odd pitch keeps the 8 rows on 8 banks
    const int pitch = cu * 128 + 64;
    float *sums = reinterpret_cast<float *>(total + nt * NB * 32);
    uint4 *zeros = reinterpret_cast<uint4 *>(sums + cu * SETS * C);
    __half2 *pairs = reinterpret_cast<__half2 *>(zeros + 8);
    uint8_t *act = reinterpret_cast<uint8_t *>(pairs) + ((nt * 16 * sp * 4 + 15) & ~15);

    const int64_t row_words = (int64_t)p.K * BITS / 32;
    const uint32_t shift = BITS & 1 ? (uint32_t)(q & 1) * 16u : 0u;
    for (int u0 = 0; u0 < U; u0 += cu) {
        const int n = U - u0 < cu ? U - u0 : cu;  // units of this chunk
        const int total_units = nt * n;
        const int beg = total_units * warp / kWarps, end = total_units * (warp + 1) / kWarps;
        int t = beg / n, u = beg - t * n;

        // codes: pointers of the loads in flight, one unit after the other
        const int64_t row0 = (int64_t)ps.e * p.R + (int64_t)(ps.tile0 + t) * (PAIRS ? 8 : 16) + g;
        const int64_t off = row0 * row_words + (int64_t)(u0 + u) * (2 * BITS) + BITS * q / 2;
        const uint32_t *pa = p.w0 + off;
        const uint32_t *pb = (PAIRS ? p.w1 : p.w0 + 8 * row_words) + off;
        const int64_t jump = (PAIRS ? 8 : 16) * row_words - (int64_t)n * (2 * BITS);
        int pu = u;
        uint32_t wa[AHEAD][NW], wb[AHEAD][NW];
        auto fetch = [&](uint32_t(&a)[NW], uint32_t(&b)[NW]) {
            load_codes<BITS>(pa, a);
            load_codes<BITS>(pb, b);
            pa += 2 * BITS;
            pb += 2 * BITS;
            if (++pu == n) {
                pu = 0;
                pa += jump;
                pb += jump;
            }
        };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (beg + i < end) fetch(wa[i], wb[i]);

        if (wait && u0 == 0) grid_dependency_wait();
        if (u0 == 0 && tid < 32) sh.peak[tid] = 0u;
        __syncthreads();  // the last chunk's or pass's readers are done

        // (scale, bias) of the pass's rows
        const int g0 = (int)((int64_t)u0 * 64 / p.group), ng = (n * 64 + p.group - 1) / p.group;
        for (int i = tid; i < nt * 16 * ng; i += kThreads) {
            const int row = i / ng, k = i - row * ng, r = row & 15;
            const bool second = PAIRS && r >= 8;
            const int64_t at =
                ((int64_t)ps.e * p.R + (int64_t)(ps.tile0 + (row >> 4)) * (PAIRS ? 8 : 16) +
                 (PAIRS ? r & 7 : r)) * groups + g0 + k;
            const __half s = static_cast<const __half *>(second ? p.s1 : p.s0)[at];
            const __half b = static_cast<const __half *>(second ? p.b1 : p.b0)[at];
            pairs[row * sp + k] = __halves2half2(s, b);
        }
        // the columns' largest magnitudes
        if (u0 == 0) {
            for (int i = tid; i < ps.ncols * U * 4; i += kThreads) {
                const int c = i / (U * 4);
                const int entry = sh.list[ps.col0 + c];
                float v[16];
                source16<PAIRS>(p, (size_t)(PAIRS ? entry / p.top : entry) * p.K +
                                       (size_t)(i - c * U * 4) * 16, v);
                float m = 0.f;
#pragma unroll
                for (int k = 0; k < 16; ++k) m = fmaxf(m, fabsf(v[k]));
                atomicMax(&sh.peak[c], __float_as_uint(m));
            }
            if (tid < 8) zeros[tid] = make_uint4(0u, 0u, 0u, 0u);
            __syncthreads();
        }
        // the columns in MMA order, with their group sums
        for (int i = tid; i < ps.ncols * n * 4; i += kThreads) {
            const int c = i / (n * 4), r = i - c * n * 4, uu = r >> 2, qq = r & 3;
            const int entry = sh.list[ps.col0 + c];
            float v[16];
            source16<PAIRS>(p, (size_t)(PAIRS ? entry / p.top : entry) * p.K +
                                   (size_t)(u0 * 4 + r) * 16, v);
            // 2^up puts the largest magnitude into [2^14, 2^15)
            const int ex = (int)(sh.peak[c] >> 23);
            int up = ex == 0 || ex == 255 ? 0 : 14 + 127 - ex;
            up = up > 100 ? 100 : up;
            const float f = __int_as_float((127 + up) << 23);
            if (r == 0) sh.undo[c] = __int_as_float((127 - up) << 23);
            float s = 0.f;
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                v[k] *= f;
                s += __half2float(__float2half_rn(v[k]));
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float down = 1.f / (float)(1 << Order<BITS>::pre(k));
                o[k] = pack_half2(v[Order<BITS>::lo(k)] * down, v[Order<BITS>::hi(k)] * down);
            }
            uint4 *dst = reinterpret_cast<uint4 *>(act + (size_t)c * pitch + uu * 128) + qq;
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[4] = make_uint4(o[4], o[5], o[6], o[7]);
            const uint32_t quad = 0xFu << (lane & ~3);  // a unit's four lanes come together
            s += __shfl_xor_sync(quad, s, 1);
            if (!G32) s += __shfl_xor_sync(quad, s, 2);
            if (G32 ? (qq & 1) == 0 : qq == 0)
                sums[(uu * SETS + (G32 ? qq >> 1 : 0)) * C + c] = s * 5.9604644775390625e-08f;
        }
        __syncthreads();

        const uint8_t *bp[NB][SETS];
        uint32_t step[SETS];
#pragma unroll
        for (int h = 0; h < SETS; ++h) {
            const bool mine = !G32 || (q >> 1) == h;
            step[h] = mine ? 128u : 0u;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int c = nb * 8 + g;
                bp[nb][h] = mine ? act + (size_t)(c < ps.ncols ? c : 0) * pitch + q * 16
                                 : reinterpret_cast<const uint8_t *>(zeros);
            }
        }
        float acc[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nb][i] = 0.f;

        auto flush = [&]() {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                slots[((t + warp) * NB + nb) * 32 + lane] =
                    make_float4(acc[nb][0], acc[nb][1], acc[nb][2], acc[nb][3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[nb][i] = 0.f;
            }
        };
        for (int base = beg; base < end; base += AHEAD) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (base + i < end) {
                    uint32_t ra[8], rb[8];
                    decode<BITS>(wa[i], shift, ra);
                    decode<BITS>(wb[i], shift, rb);
                    if (base + i + AHEAD < end) fetch(wa[i], wb[i]);
#pragma unroll
                    for (int h = 0; h < SETS; ++h) {
                        const int gi = p.group == 128 ? u >> 1 : u * SETS + h;
                        const float2 sa = __half22float2(pairs[(t * 16 + g) * sp + gi]);
                        const float2 sb = __half22float2(pairs[(t * 16 + 8 + g) * sp + gi]);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            const uint8_t *b = bp[nb][h] + u * step[h];
                            const uint4 x = *reinterpret_cast<const uint4 *>(b);
                            const uint4 y = *reinterpret_cast<const uint4 *>(b + 64);
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
                            mma(d, ra[0], rb[0], ra[1], rb[1], x.x, x.y);
                            mma(d, ra[2], rb[2], ra[3], rb[3], x.z, x.w);
                            mma(d, ra[4], rb[4], ra[5], rb[5], y.x, y.y);
                            mma(d, ra[6], rb[6], ra[7], rb[7], y.z, y.w);
                            const float2 s = *reinterpret_cast<const float2 *>(
                                sums + (u * SETS + h) * C + nb * 8 + 2 * q);
                            acc[nb][0] = fmaf(sa.x, d[0], fmaf(sa.y, s.x, acc[nb][0]));
                            acc[nb][1] = fmaf(sa.x, d[1], fmaf(sa.y, s.y, acc[nb][1]));
                            acc[nb][2] = fmaf(sb.x, d[2], fmaf(sb.y, s.x, acc[nb][2]));
                            acc[nb][3] = fmaf(sb.x, d[3], fmaf(sb.y, s.y, acc[nb][3]));
                        }
                    }
                    if (++u == n) {
                        flush();
                        u = 0;
                        ++t;
                    }
                }
            }
        }
        if (u != 0 && beg < end) flush();
        __syncthreads();

        // the tiles' sums, in warp order; after the last chunk the results
        for (int i = tid; i < nt * NB * 32; i += kThreads) {
            const int tt = i / (NB * 32), nb = i / 32 % NB, ln = i & 31;
            float4 s = u0 == 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : total[i];
            for (int w = 0; w < kWarps; ++w) {
                const int b = max(total_units * w / kWarps, tt * n);
                const int e = min(total_units * (w + 1) / kWarps, (tt + 1) * n);
                if (b < e) {
                    const float4 v = slots[((tt + w) * NB + nb) * 32 + ln];
                    s.x += v.x;
                    s.y += v.y;
                    s.z += v.z;
                    s.w += v.w;
                }
            }
            if (u0 + n < U) {
                total[i] = s;
                continue;
            }
            const int row = (ps.tile0 + tt) * (PAIRS ? 8 : 16) + (ln >> 2);
            const float part[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = nb * 8 + 2 * (ln & 3) + j;
                if (c >= ps.ncols) continue;
                const float a = part[j] * 16777216.f * sh.undo[c];
                const float b = part[2 + j] * 16777216.f * sh.undo[c];
                float *to = p.dst + (size_t)sh.list[ps.col0 + c] * p.R + row;
                if constexpr (PAIRS) {
                    *to = a / (1.f + expf(-a)) * b;
                } else {
                    to[0] = a;
                    to[8] = b;
                }
            }
        }
    }
}

template <int BITS, bool G32, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 2) moe_kernel(const __grid_constant__ MoeParams p) {
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ Shared sh;
    // the ids are there before this grid's predecessor starts (down), or are
    // what it writes (gate and up)
    if (PAIRS) {
        grid_dependency_wait();
        launch_dependents();
    }
    plan(p, sh);
    const int per = p.R / (PAIRS ? 8 : 16);
    const int64_t tiles = (int64_t)sh.busy * per;
    int64_t lo = tiles * blockIdx.x / gridDim.x;
    const int64_t hi = tiles * (blockIdx.x + 1) / gridDim.x;
    bool wait = !PAIRS;
    if (wait && lo >= hi) grid_dependency_wait();
    int last = -1;
    while (lo < hi) {
        const int a = (int)(lo / per);
        Pass ps;
        ps.e = sh.act[a];
        ps.tile0 = (int)(lo - (int64_t)a * per);
        int left = per - ps.tile0;
        if (hi - lo < left) left = (int)(hi - lo);
        if (ps.e != last) list_entries(p, ps.e, sh);
        last = ps.e;
        const int count = sh.count[ps.e];
        // as many tiles as leave the whole of K in one chunk, else a few
        const int most = count < 32 ? count : 32, nb = most <= 8 ? 1 : most <= 16 ? 2 : 4;
        ps.nt = left < kMaxTiles ? left : kMaxTiles;
        while (ps.nt > 1 && units_that_fit(ps.nt, most, nb, G32 ? 2 : 1) < p.K / 64) --ps.nt;
        if (units_that_fit(ps.nt, most, nb, G32 ? 2 : 1) < p.K / 64) {
            ps.nt = nb == 4 ? 4 : 8;
            if (left < ps.nt) ps.nt = left;
        }
        for (ps.col0 = 0; ps.col0 < count; ps.col0 += 32) {
            ps.ncols = count - ps.col0 < 32 ? count - ps.col0 : 32;
            if (ps.ncols <= 8)
                run_pass<BITS, G32, PAIRS, 1>(p, ps, sh, dyn, wait);
            else if (ps.ncols <= 16)
                run_pass<BITS, G32, PAIRS, 2>(p, ps, sh, dyn, wait);
            else
                run_pass<BITS, G32, PAIRS, 4>(p, ps, sh, dyn, wait);
            wait = false;
        }
        lo += ps.nt;
    }
}

// The grid: two CTAs an SM, each with an even run of tiles.
template <int BITS, bool G32, bool PAIRS>
cudaError_t launch_one(const MoeParams &p, cudaStream_t stream) {
    auto *kern = moe_kernel<BITS, G32, PAIRS>;
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

template <int BITS>
cudaError_t launch(const MoeParams &p, bool pairs, cudaStream_t stream) {
    if (p.group == 32)
        return pairs ? launch_one<BITS, true, true>(p, stream)
                     : launch_one<BITS, true, false>(p, stream);
    return pairs ? launch_one<BITS, false, true>(p, stream)
                 : launch_one<BITS, false, false>(p, stream);
}

}  // namespace moe_detail
}  // namespace aq
