// The batch attention's kernel for few rows a tile (a sequence's own keys,
// and shared keys of small groups): warp MMA, codes as they lie in the cache.
//
//   S^T[key][row] = scale_k (codes_k . q') + bias_k sum(q)        (per group)
//   O^T[d][row]  += codes_v[d][key] (p scale_v)[key][row],  + sum p bias_v
//
// The keys are the MMA's 16 rows and the query rows its 8 columns, so that a
// decode step's few query rows a KV head (R tokens x heads) fill the MMA and
// each code is read and converted once for all of them (NB blocks of 8
// columns share the converted fragment).  K codes enter as exact fp16
// subnormals (code * 2^-24, or 2^-20 where a nibble sits at bit 4), scale and
// bias in fp32 on the sums.  V codes enter less the middle code (8 or 128,
// exact): sums of codes as they are grow with the number of keys, and the
// tensor core's accumulation, which truncates, then loses what is left of
// them after the bias (0.6 % of the output over 33,000 keys of 8 bits).
// p * scale_v * 2^ev enters as fp16 (2^-11 relative; ev a power of two a warp
// lowers as larger scales appear).
//
// Every warp works alone: it takes an even run of the call's tiles (16 or 32
// keys of one KV head, see aq_batch.cuh), streams them through a ring of its
// own in shared memory with 16-byte cp.async, the page numbers one tile ahead,
// and writes its own partial results - no CTA barrier after the plan, and no
// piece so short that others wait for it.  Rows in the ring are padded so that
// the fragment reads fall in distinct banks.
//
// What bounds it: the cache's bytes are 2 D bits/8 + 8 D/group a key and head
// (30.8 us for 24 ragged sequences of up to 8k rows, 8 heads of 256 at 4 bits)
// and it takes 61 us of the call's 72.  Issue slots are 56 % taken and DRAM is
// at 46 %; the registers (242 a lane) leave 8 warps an SM, so that neither
// hides the other's latency: fewer query rows than the MMA's eight columns
// make each code's unpacking dear.
#pragma once

#include "aq_batch.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace aq {

template <int BITS, int D, int GROUP, int NB>
struct Own {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRows = 8 * NB;               // query rows a tile
    static constexpr int kRB = D * BITS / 8;           // bytes of a row's codes
    static constexpr int kG = D / GROUP;
    static constexpr int kGB = GROUP * BITS / 8;       // bytes of a group's codes
    // 16-key blocks a tile: two where a row is short or its codes cost the most
    // work a byte (24 sequences of up to 8k rows of 256 at 4 bits: 80 us with
    // one, 72 with two, 75 with one at 168 registers and three CTAs an SM; 128-byte rows at 8 bits: 182 and 187 us with the shared part)
    static constexpr int kBlk = kRB <= 64 || (kRB == 128 && BITS == 4) ? 2 : 1;
    static constexpr int kKeys = 16 * kBlk;            // keys a tile
    static constexpr int kKS = kRB + (kRB >= 64 ? 32 : 0);  // K row stride in the ring
    static constexpr int kVS = kRB + 16;               // V row stride
    static constexpr int kSB = kKeys * kG * 4;         // bytes of a tile's K (or V) pairs
    static constexpr int kStage = kKeys * (kKS + kVS) + 2 * kSB;
    static constexpr int kStages = kStage <= 4096 ? 3 : 2;
    static constexpr int kSteps = GROUP / 16;
    // the q' fragments stay in registers unless they are 64 or more of them
    static constexpr bool kQRegs = NB * D <= 256;
    static constexpr int kFrag = kQRegs ? 0 : NB * (D / 16) * 32 * 8;
    static constexpr int kSums = 4 * kRows * kG;       // sums of q
    static constexpr int kWarpBytes = (kStages * kStage + kFrag + kSums + 15) / 16 * 16;
    static constexpr int kSmem = kWarps * kWarpBytes;
};

template <int N>
__device__ __forceinline__ void own_words(const uint8_t *p, uint32_t (&w)[N / 4 > 0 ? N / 4 : 1]) {
    if constexpr (N == 2) {
        w[0] = *reinterpret_cast<const uint16_t *>(p);
    } else if constexpr (N == 4) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (N == 8) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        static_assert(N == 16, "");
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    }
}

__device__ __forceinline__ uint32_t own_transpose(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ void own_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two fp16 codes at the low bits of each half, less the middle code: exact
// (1024 + code, then the subtraction).
__device__ __forceinline__ uint32_t centred(uint32_t codes, float middle) {
    const uint32_t u = codes | 0x64006400u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&u),
                              __half2half2(__float2half_rn(middle)));
    return *reinterpret_cast<const uint32_t *>(&r);
}

template <int BITS, int D, int GROUP, int NB>
__global__ void __launch_bounds__(128) own_kernel(const __grid_constant__ BatchParams p) {
    using S = Own<BITS, D, GROUP, NB>;
    constexpr int G = S::kG, BLK = S::kBlk;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gid = lane >> 2, t = lane & 3;
    uint8_t *my = smem + warp * S::kWarpBytes;
    uint2 *qfrag = reinterpret_cast<uint2 *>(my + S::kStages * S::kStage);
    float *qs2 = reinterpret_cast<float *>(my + S::kStages * S::kStage + S::kFrag);  // [rows][G]

    // After shared_kernel, which has seen the plan complete before it let this
    // kernel start, there is nothing to wait for: its pieces are other slots.
    // (What earlier kernels wrote is then read past L1, which may be older.)
    if (!p.shared_tc) grid_dependency_wait();
    launch_dependents();
    const int me = (int)blockIdx.x * S::kWarps + warp;
    const int4 head = __ldcg(reinterpret_cast<const int4 *>(p.head));  // per, tiles, ..
    const int per = head.x, LR = p.L * p.R;
    // (long long: runs past the last tile are empty, wherever they start)
    long long u64 = (long long)me * per;
    const int end = (int)min((long long)head.y, u64 + per);
    int u = (int)min(u64, (long long)end), at = u < end ? __ldcg(p.runs + me) : 0;
    uint32_t outside = 0;

    while (u < end) {
        // the segment (one KV head and row tile of a group's or row's keys) of
        // tile u, and this run's part of it
        Piece w;
        const bool is_shared = at < 0;
        int base, tiles, rows, first, step;
        if (is_shared) {
            const PlanGroup g = plan_load(p.groups - 1 - at);
            base = g.at;
            tiles = g.pieces;
            rows = g.rows * LR;
            step = g.rows;
            w.row = g.lead;
            w.b0 = g.first;
            w.k0 = 0;
            w.k1 = g.len;
            w.slot0 = g.slot;
        } else {
            const PlanRow b = plan_load(p.rows + at);
            base = b.at;
            tiles = b.tiles;
            rows = LR;
            step = 1;
            w.row = w.b0 = at;
            w.k0 = b.k0;
            w.k1 = b.k1;
            w.slot0 = b.slot;
        }
        const int rt = ceil_div(rows, S::kRows);
        if (u - base >= tiles * p.c.KV * rt) {  // the next one (empty ones are passed over)
            at = is_shared && at > -p.G ? at - 1 : is_shared ? 0 : at + 1;
            continue;
        }
        const int seg = (u - base) / tiles, off = u - base - seg * tiles;
        const int n = min(tiles - off, end - u);
        first = w.k0 / S::kKeys + off;
        w.kv = seg / rt;
        w.r0 = (seg - w.kv * rt) * S::kRows;
        w.rows = min(S::kRows, rows - w.r0);
        // a slot (a sequence) for each run that touches the segment
        w.slot0 += (me - (base + seg * tiles) / per) * step;
        const int row_len = w.k1;
        w.k0 = max(w.k0, first * S::kKeys);
        w.k1 = min(w.k1, (first + n) * S::kKeys);
        u += n;
        const int tile0 = first, tile1 = first + n;
        const int32_t *trow = p.table + (int64_t)w.row * p.max_pages;
        // the page of each 16-key block of a tile, in lane = block
        auto page_of = [&](int tile) -> int {
            int id = -1;
            const int key = tile * S::kKeys + 16 * (lane & (BLK - 1));
            if (tile < tile1 && key < w.k1) {
                id = __ldcg(trow + (key >> p.c.page_log2));
                if (id < 0 || id >= p.c.n_pages) {
                    id = -1;
                    outside = 1;
                }
            }
            return id;
        };
        auto load = [&](int tile, int stage, int ids) {
            uint8_t *st = my + stage * S::kStage;
            const int key0 = tile * S::kKeys;
#pragma unroll
            for (int b = 0; b < BLK; ++b) {
                const int id = __shfl_sync(~0u, ids, b);
                const int slot = (key0 + 16 * b) & (p.c.page - 1);
                const uint32_t ok = id >= 0 ? 16u : 0u;
                const uint8_t *rec = p.layer + max(id, 0) * p.c.page_bytes + w.kv * p.c.rec;
                const uint8_t *kc = rec + slot * S::kRB, *vc = kc + p.c.side_codes;
                const uint8_t *ks = rec + 2 * (int64_t)p.c.side_codes + slot * (4 * G);
                const uint8_t *vs = ks + p.c.side_sb;
                constexpr int PR = S::kRB / 16;  // 16-byte pieces a row
#pragma unroll
                for (int i = 0; i < 16 * PR / 32 + (16 * PR % 32 != 0); ++i) {
                    const int x = lane + 32 * i;
                    if (16 * PR % 32 == 0 || x < 16 * PR) {
                        const int row = 16 * b + x / PR, col = 16 * (x % PR);
                        cp_async16(st + row * S::kKS + col, kc + 16 * x, ok);
                        cp_async16(st + S::kKeys * S::kKS + row * S::kVS + col, vc + 16 * x, ok);
                    }
                }
                constexpr int NS = 16 * G * 4 / 16;  // pieces of 16 keys' pairs
                uint8_t *sk = st + S::kKeys * (S::kKS + S::kVS) + b * 16 * NS;
                for (int x = lane; x < 2 * NS; x += 32)
                    cp_async16(x < NS ? sk + 16 * x : sk + S::kSB + 16 * (x - NS),
                               x < NS ? ks + 16 * x : vs + 16 * (x - NS), ok);
            }
        };


        // the first tiles are under way while q' is made
        int ids = page_of(tile0);
#pragma unroll
        for (int s = 0; s < S::kStages - 1; ++s) {
            const int nxt = page_of(tile0 + s + 1);
            if (tile0 + s < tile1) load(tile0 + s, s, ids);
            cp_async_commit();
            ids = nxt;
        }

        // ---------------------------------------------------------------- q'
        // Lane (gid, t) holds D / 4 values of row gid: those that meet the
        // codes it reads.  q' = q * 2^e a row, in fp16; at 4 bits the values
        // of codes at bit 4 carry another 2^-4.
        uint2 qr[S::kQRegs ? NB * (D / 16) : 1];
        int lim[2 * NB], lim_min = w.k1;
        float qc[2 * NB];
        __syncwarp();
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int r = nb * 8 + gid;
            uint4 raw[D / 32];
            const uint4 *src = nullptr;
            if (r < w.rows) src = reinterpret_cast<const uint4 *>(q_row(p, w, r));
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < GROUP / 32; ++i)
                    raw[g * (GROUP / 32) + i] =
                        src ? __ldcg(src + g * (GROUP / 8) + t * (GROUP / 32) + i)
                            : make_uint4(0u, 0u, 0u, 0u);
            float mx = 0.f;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < GROUP / 32; ++i) {
                    const uint4 x = raw[g * (GROUP / 32) + i];
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float f = q_float(p, (uint16_t)(xs[k / 2] >> (16 * (k & 1))));
                        mx = fmaxf(mx, fabsf(f));
                        sum += f;
                    }
                }
                sum += __shfl_xor_sync(~0u, sum, 1);
                sum += __shfl_xor_sync(~0u, sum, 2);
                if (t == 0) qs2[r * G + g] = sum * p.scale2;
            }
            mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
            const int e = batch_exp(mx);
            const float sc = batch_pow2(e);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t xs[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                float f[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    f[k] = q_float(p, (uint16_t)(xs[k / 2] >> (16 * (k & 1)))) * sc;
                uint2 fr[2];
                if constexpr (BITS == 4) {
                    fr[0] = make_uint2(pack_half2(f[0], f[4]),
                                       pack_half2(f[1] * 0.0625f, f[5] * 0.0625f));
                    fr[1] = make_uint2(pack_half2(f[2], f[6]),
                                       pack_half2(f[3] * 0.0625f, f[7] * 0.0625f));
                } else {
                    fr[0] = make_uint2(pack_half2(f[0], f[2]), pack_half2(f[1], f[3]));
                    fr[1] = make_uint2(pack_half2(f[4], f[6]), pack_half2(f[5], f[7]));
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if constexpr (S::kQRegs)
                        qr[nb * (D / 16) + 2 * i + k] = fr[k];
                    else
                        qfrag[(nb * (D / 16) + 2 * i + k) * 32 + lane] = fr[k];
                }
            }
            // factors and limits of the columns this lane has: rows 2t, 2t + 1
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = 2 * nb + i, rc = nb * 8 + 2 * t + i;
                qc[c] = batch_pow2(24 - __shfl_sync(~0u, e, (2 * t + i) * 4)) * p.scale2;
                // keys at and past the limit are not seen by the row
                const int l = (w.r0 + rc) % (p.L * p.R) / p.R;
                lim[c] = rc >= w.rows ? 0
                         : is_shared  ? w.k1
                                      : min(w.k1, row_len - (p.L - 1 - l));
                if (rc < w.rows) lim_min = min(lim_min, lim[c]);
            }
        }
        lim_min = __reduce_min_sync(~0u, lim_min);
        __syncwarp();

        // --------------------------------------------------------- the keys
        float m2[2 * NB], l[2 * NB], bt[2 * NB][G], O[D / 16][NB][4];
        int ev = 127;
#pragma unroll
        for (int c = 0; c < 2 * NB; ++c) {
            m2[c] = -INFINITY;
            l[c] = 0.f;
#pragma unroll
            for (int g = 0; g < G; ++g) bt[c][g] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
                O[i][nb][0] = O[i][nb][1] = O[i][nb][2] = O[i][nb][3] = 0.f;
        int stage = 0;
#pragma unroll 1
        for (int tile = tile0; tile < tile1; ++tile) {
            {
                const int ahead = tile + S::kStages - 1;
                const int nxt = page_of(ahead + 1);
                const int into = stage == 0 ? S::kStages - 1 : stage - 1;
                if (ahead < tile1) load(ahead, into, ids);
                cp_async_commit();
                ids = nxt;
            }
            cp_async_wait<S::kStages - 1>();
            __syncwarp();
            const uint8_t *kst = my + stage * S::kStage;
            const uint8_t *vst = kst + S::kKeys * S::kKS;
            const __half2 *ksb = reinterpret_cast<const __half2 *>(vst + S::kKeys * S::kVS);
            const __half2 *vsb = ksb + S::kSB / 4;
            const int key0 = tile * S::kKeys;

            // ------------------------------------------------------ scores
            float s[BLK][NB][4];
#pragma unroll
            for (int b = 0; b < BLK; ++b) {
                float t2[NB][4];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[b][nb][i] = t2[nb][i] = 0.f;
                const int ra = 16 * b + gid, rb = ra + 8;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    constexpr int NBY = S::kGB / 4;  // bytes a lane takes of a group
                    constexpr int PC = NBY < 8 ? NBY : 8;
                    float acc[NB][4];
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        acc[nb][0] = acc[nb][1] = acc[nb][2] = acc[nb][3] = 0.f;
#pragma unroll
                    for (int c = 0; c < NBY / PC; ++c) {
                        uint32_t wa[PC / 4], wb[PC / 4];
                        const int byte = g * S::kGB + t * NBY + c * PC;
                        own_words<PC>(kst + ra * S::kKS + byte, wa);
                        own_words<PC>(kst + rb * S::kKS + byte, wb);
#pragma unroll
                        for (int j = 0; j < PC / 4; ++j) {
                            constexpr int KW = BITS == 4 ? 2 : 1;  // k-steps a word
                            uint32_t Ra[2 * KW], Rb[2 * KW];
                            if constexpr (BITS == 4) {
                                const uint32_t va = wa[j] >> 8, vb = wb[j] >> 8;
                                Ra[0] = wa[j] & 0x000F000Fu;
                                Ra[1] = wa[j] & 0x00F000F0u;
                                Ra[2] = va & 0x000F000Fu;
                                Ra[3] = va & 0x00F000F0u;
                                Rb[0] = wb[j] & 0x000F000Fu;
                                Rb[1] = wb[j] & 0x00F000F0u;
                                Rb[2] = vb & 0x000F000Fu;
                                Rb[3] = vb & 0x00F000F0u;
                            } else {
                                Ra[0] = wa[j] & 0x00FF00FFu;
                                Ra[1] = (wa[j] >> 8) & 0x00FF00FFu;
                                Rb[0] = wb[j] & 0x00FF00FFu;
                                Rb[1] = (wb[j] >> 8) & 0x00FF00FFu;
                            }
#pragma unroll
                            for (int k = 0; k < KW; ++k) {
                                const int step = (c * (PC / 4) + j) * KW + k;
                                const uint32_t a[4] = {Ra[2 * k], Rb[2 * k], Ra[2 * k + 1],
                                                       Rb[2 * k + 1]};
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb) {
                                    const int at = nb * (D / 16) + g * S::kSteps + step;
                                    const uint2 bq = S::kQRegs ? qr[at] : qfrag[at * 32 + lane];
                                    own_mma(acc[nb], a, bq.x, bq.y);
                                }
                            }
                        }
                    }
                    const float2 sa = __half22float2(ksb[ra * G + g]);
                    const float2 sb = __half22float2(ksb[rb * G + g]);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const float q0 = qs2[(nb * 8 + 2 * t) * G + g];
                        const float q1 = qs2[(nb * 8 + 2 * t + 1) * G + g];
                        s[b][nb][0] = fmaf(sa.x, acc[nb][0], s[b][nb][0]);
                        s[b][nb][1] = fmaf(sa.x, acc[nb][1], s[b][nb][1]);
                        s[b][nb][2] = fmaf(sb.x, acc[nb][2], s[b][nb][2]);
                        s[b][nb][3] = fmaf(sb.x, acc[nb][3], s[b][nb][3]);
                        t2[nb][0] = fmaf(sa.y, q0, t2[nb][0]);
                        t2[nb][1] = fmaf(sa.y, q1, t2[nb][1]);
                        t2[nb][2] = fmaf(sb.y, q0, t2[nb][2]);
                        t2[nb][3] = fmaf(sb.y, q1, t2[nb][3]);
                    }
                }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[b][nb][i] = fmaf(qc[2 * nb + (i & 1)], s[b][nb][i], t2[nb][i]);
            }
            // keys that a row does not see: weight 0, whatever the cache holds
            const bool edge = key0 < w.k0 || key0 + S::kKeys > lim_min;
            if (edge) {
#pragma unroll
                for (int b = 0; b < BLK; ++b)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = key0 + 16 * b + gid + 8 * (i >> 1);
                            if (key < w.k0 || key >= lim[2 * nb + (i & 1)])
                                s[b][nb][i] = -INFINITY;
                        }
            }

            // ------------------------------------- online softmax (base 2)
            float vmx = 0.f;
            float2 va[BLK][G], vb[BLK][G];
#pragma unroll
            for (int b = 0; b < BLK; ++b)
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const int ra = 16 * b + gid, rb = ra + 8;
                    va[b][g] = __half22float2(vsb[ra * G + g]);
                    vb[b][g] = __half22float2(vsb[rb * G + g]);
                    if (edge) {  // pairs of keys that nobody sees may be anything
                        if (key0 + ra < w.k0 || key0 + ra >= w.k1) va[b][g] = make_float2(0.f, 0.f);
                        if (key0 + rb < w.k0 || key0 + rb >= w.k1) vb[b][g] = make_float2(0.f, 0.f);
                    }
                    float xa = fabsf(va[b][g].x), xb = fabsf(vb[b][g].x);
                    if (edge) {  // nor does one that only some rows see set ev unless finite
                        if (!(xa <= 65504.f)) xa = 0.f;
                        if (!(xb <= 65504.f)) xb = 0.f;
                    }
                    vmx = fmaxf(vmx, fmaxf(xa, xb));
                }
            vmx = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(vmx)));
            const int ev_new = min(ev, batch_exp(vmx));
            const float rv = ev_new - ev < -126 ? 0.f : batch_pow2(ev_new - ev);
            ev = ev_new;
            const float vsc = batch_pow2(ev);
            float f[2 * NB];
            bool changed = rv != 1.f;
#pragma unroll
            for (int c = 0; c < 2 * NB; ++c) {
                const int nb = c >> 1, i = c & 1;
                float mx = fmaxf(s[0][nb][i], s[0][nb][2 + i]);
#pragma unroll
                for (int b = 1; b < BLK; ++b)
                    mx = fmaxf(mx, fmaxf(s[b][nb][i], s[b][nb][2 + i]));
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
                const float mn = fmaxf(m2[c], mx);
                // nothing seen yet: keep the weights at 2^-inf = 0
                const float ref = mn == -INFINITY ? 0.f : mn;
                f[c] = batch_ex2(m2[c] - ref);
                m2[c] = mn;
                changed |= f[c] != 1.f;
                float ls = 0.f;
#pragma unroll
                for (int b = 0; b < BLK; ++b) {
                    s[b][nb][i] = batch_ex2(s[b][nb][i] - ref);
                    s[b][nb][2 + i] = batch_ex2(s[b][nb][2 + i] - ref);
                    ls += s[b][nb][i] + s[b][nb][2 + i];
                }
                l[c] = fmaf(l[c], f[c], ls);
            }
            if (__any_sync(~0u, changed)) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const float o0 = f[2 * nb] * rv, o1 = f[2 * nb + 1] * rv;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        O[i][nb][0] *= o0;
                        O[i][nb][1] *= o1;
                        O[i][nb][2] *= o0;
                        O[i][nb][3] *= o1;
                    }
                }
#pragma unroll
                for (int c = 0; c < 2 * NB; ++c)
#pragma unroll
                    for (int g = 0; g < G; ++g) bt[c][g] *= f[c];
            }

            // ------------------------------------------------------ values
#pragma unroll
            for (int g = 0; g < G; ++g) {
#pragma unroll
                for (int b = 0; b < BLK; ++b) {
                    uint32_t pb[NB][2];
                    const float xa = va[b][g].x * vsc, xb = vb[b][g].x * vsc;
                    // the bias of centred codes: bias + middle code * scale
                    constexpr float kMid = BITS == 4 ? 8.f : 128.f;
                    const float ya = fmaf(kMid, va[b][g].x, va[b][g].y);
                    const float yb = fmaf(kMid, vb[b][g].x, vb[b][g].y);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        float w0 = s[b][nb][0] * xa, w1 = s[b][nb][1] * xa;
                        float w2 = s[b][nb][2] * xb, w3 = s[b][nb][3] * xb;
                        float c0 = s[b][nb][0] * ya, c1 = s[b][nb][1] * ya;
                        float c2 = s[b][nb][2] * yb, c3 = s[b][nb][3] * yb;
                        if (edge) {
                            // a token that some of the tile's rows do not see: its
                            // pair must not reach them even where it is not finite
                            const int ka = key0 + 16 * b + gid, kb = ka + 8;
                            if (ka >= lim[2 * nb]) w0 = c0 = 0.f;
                            if (ka >= lim[2 * nb + 1]) w1 = c1 = 0.f;
                            if (kb >= lim[2 * nb]) w2 = c2 = 0.f;
                            if (kb >= lim[2 * nb + 1]) w3 = c3 = 0.f;
                        }
                        bt[2 * nb][g] += c0 + c2;
                        bt[2 * nb + 1][g] += c1 + c3;
                        pb[nb][0] = own_transpose(pack_half2(w0, w1));
                        pb[nb][1] = own_transpose(pack_half2(w2, w3));
                    }
                    constexpr int NV = S::kGB / 8;  // bytes a lane takes of a group
                    constexpr int PC = NV < 8 ? NV : 8;
                    constexpr int NW = PC >= 4 ? PC / 4 : 1;
                    const uint8_t *vrow = vst + (16 * b + 2 * t) * S::kVS + g * S::kGB + gid * NV;
#pragma unroll
                    for (int c = 0; c < NV / PC; ++c) {
                        uint32_t w0[NW], w1[NW], w8[NW], w9[NW];
                        own_words<PC>(vrow + c * PC, w0);
                        own_words<PC>(vrow + S::kVS + c * PC, w1);
                        own_words<PC>(vrow + 8 * S::kVS + c * PC, w8);
                        own_words<PC>(vrow + 9 * S::kVS + c * PC, w9);
                        constexpr int MT = PC * 8 / BITS / 2;  // M-tiles of these bytes
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            uint32_t a[4];
                            if constexpr (BITS == 4) {
                                const int wi = m / 4, bi = m % 4;
                                const uint32_t sel = (uint32_t)bi | ((uint32_t)(4 + bi) << 8);
                                const uint32_t x = prmt(w0[wi], w1[wi], sel);
                                const uint32_t y = prmt(w8[wi], w9[wi], sel);
                                a[0] = centred(x & 0x000F000Fu, 1032.f);
                                a[1] = centred(x & 0x00F000F0u, 1152.f);
                                a[2] = centred(y & 0x000F000Fu, 1032.f);
                                a[3] = centred(y & 0x00F000F0u, 1152.f);
                            } else {
                                const int wi = (2 * m) / 4, bi = (2 * m) % 4;
                                const uint32_t sl = (uint32_t)bi | ((uint32_t)(4 + bi) << 8);
                                const uint32_t sh = sl + 0x101u;
                                a[0] = centred(prmt(w0[wi], w1[wi], sl) & 0x00FF00FFu, 1152.f);
                                a[1] = centred(prmt(w0[wi], w1[wi], sh) & 0x00FF00FFu, 1152.f);
                                a[2] = centred(prmt(w8[wi], w9[wi], sl) & 0x00FF00FFu, 1152.f);
                                a[3] = centred(prmt(w8[wi], w9[wi], sh) & 0x00FF00FFu, 1152.f);
                            }
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                own_mma(O[g * S::kSteps + c * MT + m][nb], a, pb[nb][0],
                                        pb[nb][1]);
                        }
                    }
                }
            }
            __syncwarp();  // every lane is done with the stage before it is refilled
            stage = stage + 1 == S::kStages ? 0 : stage + 1;
        }
        cp_async_wait<0>();

        // ------------------------------------------------------ partial out
        const int evf = ev == 127 ? 0 : ev;
        const float fa = batch_pow2(-evf), fb = BITS == 4 ? batch_pow2(-4 - evf) : fa;
#pragma unroll
        for (int c = 0; c < 2 * NB; ++c) {
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) {
                l[c] += __shfl_xor_sync(~0u, l[c], o);
#pragma unroll
                for (int g = 0; g < G; ++g) bt[c][g] += __shfl_xor_sync(~0u, bt[c][g], o);
            }
            const int r = (c >> 1) * 8 + 2 * t + (c & 1);
            if (r >= w.rows) continue;
            const int64_t at = part_row(p, w, r);
            if (gid == 0) p.part_ml[at] = make_float2(m2[c], l[c]);
            float *o = p.part_o + at * D;
            // M-tile m of a group: values 2m, 2m + 1 of the lane's GROUP / 8
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int m = 0; m < S::kSteps; m += 2) {
                    const int x = g * S::kSteps + m, nb = c >> 1, i = c & 1;
                    *reinterpret_cast<float4 *>(o + g * GROUP + gid * (GROUP / 8) + 2 * m) =
                        make_float4(fmaf(O[x][nb][i], fa, bt[c][g]),
                                    fmaf(O[x][nb][2 + i], fb, bt[c][g]),
                                    fmaf(O[x + 1][nb][i], fa, bt[c][g]),
                                    fmaf(O[x + 1][nb][2 + i], fb, bt[c][g]));
                }
        }
        __syncwarp();
    }
    if (outside) atomicOr(p.err, ERR_BATCH_TABLE);
    // this grid's end is the end of both kernels for the one that follows
    if (p.shared_tc) grid_dependency_wait();
}

}  // namespace aq
