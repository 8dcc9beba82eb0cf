// The batch attention's kernel for keys that many rows share: tcgen05.
//
//   S[row][key] = q'[row] . k[key],  P = 2^(scale S - m),  O[row] += P v
//
// One CTA a SM takes pieces (a range of shared keys, one KV head, a tile of
// 128 or 256 query rows).  Unlike a decode step over own keys, this is bound
// by the tensor core and by what feeds it, since each key meets hundreds of
// rows: 4 D flops a (row, key) against 2 D bits/8 bytes a key.
//
//   warps 0-15   softmax: eight warps a row tile, two threads a row (half of a
//                tile's keys each).  Scores come from tensor memory, P goes
//                back there as fp16, over the scores, and is the A operand of
//                the value product.
//   warps 16-23  dequantise: codes straight from global memory into
//                registers one step ahead, fp16 k and v into shared memory in
//                the swizzled layout the tensor core reads (k as the K-major,
//                v as the MN-major operand: one layout, rows of keys).  The
//                values of a 4-bit word land in the order 0 4 1 5 2 6 3 7,
//                which q' and the output follow, so that no code is moved.
//   warp 24      issues the MMAs.
//
// Scores of two steps are in flight (two row tiles of the same keys, or the
// same row tile and two tiles of keys), so that the tensor core works on one
// while the softmax has the other.  MMAs of one thread run in issue order,
// which is what lets a step's scores overwrite the P two steps before it.
// The running maximum only moves when a row's scores exceed it by 2^8, so O
// is seldom rescaled.  Weights are taken against 2^7 below it: P up to 2^15
// still fits fp16, and weights down to 2^-21 of the maximum's keep all their
// bits (many keys behind one that outweighs them are most of an output whose
// heavy key has a small value); the sum uses the same reference.  k and v are
// rounded once to fp16 (2^-11), the few a pair of extremes puts past its
// largest number to that number (2^-10).
//
// What bounds it: 640 query rows by 8 heads over 32k shared keys of 128 at 8
// bits are 86 GFLOP, 45 us at the measured bf16 rate, and take 114 us; the
// tensor pipe is 39 % busy, the issue slots 67 %.  A slot's chain is scores ->
// maximum -> exchange -> weights -> store (about 2200 cycles for a 128-key
// tile, the two passes over the scores most of it) and then the MMAs' own
// turnaround (1950): 4200 cycles for two steps where the products alone need
// 2048.  A third slot does not fit: two tiles of scores and two of O fill
// tensor memory.  Measured and not taken: whole score rows in registers with a
// register split between the roles (the call 291 us instead of 235 at that
// point), and one pass with a guessed maximum (311 instead of 177, spills).
#include "aq_batch_shared.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <mutex>

namespace aq {
namespace {

template <int BITS, int D, int GROUP>
struct Shd {
    static constexpr int kThreads = 25 * 32;
    static constexpr int kKeys = D <= 128 ? 128 : 64;      // keys a tile
    static constexpr int kTileBytes = kKeys * D * 2;       // k or v tile
    static constexpr int kQBytes = 128 * D * 2;            // q' of one row tile
    static constexpr int kG = D / GROUP;
    static constexpr int kRB = D * BITS / 8;
    static constexpr int kWKeys = kKeys / 8;               // keys a dequantising warp takes of a tile
    static constexpr int kLane = 128 / BITS;               // values of a lane's 16 bytes
    static constexpr int kChunks = kLane / 8;              // 16-byte chunks of k or v of them
    static constexpr int kLpr = kRB / 16;                  // lanes a row
    static constexpr int kLRows = 32 / kLpr;               // rows a load
    static constexpr int kLoads = kWKeys / kLRows;
    static_assert(kLane <= GROUP && kWKeys <= 16 && kLoads >= 1, "a lane's values are of one group");
    static constexpr int kRT = D <= 128 ? 2 : 1;           // row tiles a CTA can hold
    static constexpr int kTmemO = 2 * kKeys;               // first column of O
    static_assert(kTmemO + kRT * D <= 512, "tensor memory");
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
          "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
          "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}

// Waits for the loads so far; naming the registers keeps their uses behind it.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                   "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                   "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]),
                   "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29])
                 :
                 : "memory");
    asm volatile("" : "+r"(v[30]), "+r"(v[31])::"memory");
}

// Eight columns: a load that waits, and a store.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
        : "memory");
}

// Sixteen columns: a load that waits.
__device__ __forceinline__ void tmem_ld16w(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15])
        : "memory");
}

// Descriptor of the v tile as the MN-major operand: 64-value blocks (128
// bytes a key, swizzled) block_bytes apart, groups of 8 keys 1024 bytes.
__device__ __forceinline__ uint64_t mn_desc(uint32_t smem_addr, uint32_t block_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(block_bytes >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Byte offset of 16-byte chunk c (8 values) of row r in an operand of
// `rows` rows: 64-value blocks, each row 128 bytes with its chunks swizzled.
__device__ __forceinline__ uint32_t operand_at(int rows, int r, int c) {
    return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Eight codes (a 4-bit word; two 8-bit words) to fp16 scale * code + bias,
// each rounded once; 4-bit codes in the order 0 4 1 5 2 6 3 7.
template <int BITS>
__device__ __forceinline__ uint4 values8(const uint32_t *w, __half2 s, __half2 b) {
    uint32_t o[4];
    auto put = [&](int i, uint32_t u, __half2 mul, __half2 add) {
        const __half2 q = __hfma2(*reinterpret_cast<const __half2 *>(&u), mul, add);
        const __half2 v = __hfma2(q, s, b);
        o[i] = *reinterpret_cast<const uint32_t *>(&v);
    };
    const __half2 one = __float2half2_rn(1.f), m1024 = __float2half2_rn(-1024.f);
    if constexpr (BITS == 4) {
        const __half2 sixteenth = __float2half2_rn(0.0625f), m64 = __float2half2_rn(-64.f);
        const uint32_t h = w[0] >> 8;
        put(0, (w[0] & 0x000F000Fu) | 0x64006400u, one, m1024);
        put(1, (w[0] & 0x00F000F0u) | 0x64006400u, sixteenth, m64);
        put(2, (h & 0x000F000Fu) | 0x64006400u, one, m1024);
        put(3, (h & 0x00F000F0u) | 0x64006400u, sixteenth, m64);
    } else {
        put(0, prmt(w[0], 0x64646464u, 0x4140u), one, m1024);
        put(1, prmt(w[0], 0x64646464u, 0x4342u), one, m1024);
        put(2, prmt(w[1], 0x64646464u, 0x4140u), one, m1024);
        put(3, prmt(w[1], 0x64646464u, 0x4342u), one, m1024);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Whether values of (scale, bias) pairs of at most these magnitudes could pass
// the largest fp16 number: the rounded scale of a group that holds values next
// to it, of both signs, puts the outermost code up to 2^-10 past it.
template <int BITS>
__device__ __forceinline__ bool past_fp16(__half2 most) {
    const __half top = __float2half_rn((float)((1 << BITS) - 1));
    return __hgt(__hfma(__low2half(most), top, __high2half(most)), __float2half_rn(65504.f));
}

// A lane's chunks of a k or v tile again, infinite values as the largest fp16
// number.  Hardly ever called, and kept out of the kernel's own code (tile: a
// shared-memory address): inlined, it cost 128 sequences over 32k shared
// tokens 5 us of 164 without being run, and so did generic addressing.
template <class S>
__device__ __noinline__ void clip_fp16(uint32_t tile, int row, int l) {
    const __half2 top = __float2half2_rn(65504.f);
#pragma unroll 1
    for (int i = 0; i < S::kLoads * S::kChunks; ++i) {
        const uint32_t at = tile + operand_at(S::kKeys, row + i / S::kChunks * S::kLRows,
                                              l * S::kChunks + i % S::kChunks);
        uint32_t v[4];
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(at)
                     : "memory");
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __half2 x = __hmax2(__hmin2(*reinterpret_cast<const __half2 *>(&v[k]), top), __hneg2(top));
            v[k] = *reinterpret_cast<const uint32_t *>(&x);
        }
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0]), "r"(v[1]),
                     "r"(v[2]), "r"(v[3])
                     : "memory");
    }
}

// True in one lane of a converged warp, the same one every time.  Unlike a
// test of the lane number it tells the compiler that a single thread goes on,
// which is what issuing MMAs from uniform registers wants.
__device__ __forceinline__ bool elect_lane() {
    uint32_t on;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(on));
    return on != 0;
}

// A barrier of the 256 threads of a row tile's softmax, and one that tells
// them all whether all of them say so (a wait that gave up in one warp ends
// the tile loop of all of them together, so that none misses a barrier).
__device__ __forceinline__ void row_tile_sync(int wg) {
    __syncwarp();
    asm volatile("bar.sync %0, 256;" ::"r"(1 + wg) : "memory");
}
__device__ __forceinline__ bool row_tile_all(int wg, bool me) {
    uint32_t all;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "bar.red.and.pred q, %1, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(1 + wg), "r"((uint32_t)me)
        : "memory");
    return all != 0;
}

constexpr uint32_t kNoRow = 0xffffffffu;  // of a row tile: past the piece's rows
constexpr float kMove = 8.f;  // (log2) the reference moves when a score exceeds it by more
constexpr float kRoom = 7.f;  // what weights at the reference are above 1: 2^(kMove + kRoom) fits fp16

// A bounded wait that records that it gave up.  (The other roles' waits, for
// what then never comes, run out in the same way.  A reduction by itself: with
// atomicOr the roles' registers come out such that 128 sequences over 32k
// shared tokens take 167 us instead of 165.)
__device__ __forceinline__ bool shd_wait(uint64_t *bar, uint32_t parity, uint32_t *err) {
    if (mbar_wait(bar, parity)) return true;
    asm volatile("red.relaxed.gpu.global.or.b32 [%0], %1;" ::"l"(err), "r"((uint32_t)ERR_BATCH_BASE)
                 : "memory");
    return false;
}

template <int BITS, int D, int GROUP>
__global__ void __launch_bounds__(Shd<BITS, D, GROUP>::kThreads, 1)
    shared_kernel(const __grid_constant__ BatchParams p, int row_tiles) {
    using S = Shd<BITS, D, GROUP>;
    constexpr int KT = S::kKeys;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *qs = smem;                                  // [row tiles][blocks][128][128 B]
    uint8_t *ks = qs + S::kRT * S::kQBytes;              // [2] k tiles
    uint8_t *vs = ks + 2 * S::kTileBytes;                // [2] v tiles
    float *qsc = reinterpret_cast<float *>(vs + 2 * S::kTileBytes);  // [row tiles][128]
    float *xch = qsc + S::kRT * 128;                     // [2][row tiles][halves][128]
    uint32_t *row_ids = reinterpret_cast<uint32_t *>(xch + 2 * S::kRT * 256);  // [row tiles][128]
    uint64_t *k_full = reinterpret_cast<uint64_t *>(row_ids + S::kRT * 128);
    uint64_t *k_empty = k_full + 2, *v_full = k_empty + 2, *v_empty = v_full + 2;
    uint64_t *s_full = v_empty + 2, *p_ready = s_full + 2, *o_done = p_ready + 2;
    uint64_t *q_ready = o_done + 1, *drain = q_ready + 1;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 8);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 8);
            mbar_init(&v_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 8);
        }
        mbar_init(o_done, 1);
        mbar_init(q_ready, 8 * row_tiles);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (warp == 24) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    grid_dependency_wait();
    launch_dependents();  // own_kernel needs the plan, but nothing of this kernel
    const int n_items = p.head->shared_items * p.c.KV;
    // Each role walks the pieces by itself, with running counts of pieces,
    // tiles of keys and steps (row tiles x tiles of keys).  A step's scores
    // and P have the barriers of its parity, a k or v tile those of its slot.
    // MMAs complete in issue order, so that scores of step i are behind the
    // product of step i - 2.  No barrier is ever two phases ahead of a waiter:
    // a slot's next phase needs what the waiter does next.
    uint32_t kt = 0, step = 0, piece = 0;
    bool issued = false;

    if (warp < 16) {
        // ----------------------------------------------------------- softmax
        // Two warpgroups a row tile, each half of the keys of a tile: a step's
        // scores wait for nothing longer than this, so it is the latency that
        // counts.
        const int wg = warp >> 3, half = (warp >> 2) & 1;
        constexpr int KH = KT / 2;
        uint32_t *rows = row_ids + wg * 128;
        bool ok = wg < row_tiles;
        for (int item = blockIdx.x; ok && item < n_items; item += gridDim.x, ++piece) {
            const Piece w = shared_piece(p, item);
            const int tiles = (w.k1 - w.k0 + KT - 1) / KT;
            const int rl = (warp & 3) * 32 + lane, r = wg * 128 + rl;
            // where the row tile's rows lie: (sequence x L + token) and head of each
            if (half == 0) {
                const int LR = p.L * p.R, at = w.r0 + r, i = at / LR, lr = at - i * LR, l = lr / p.R;
                rows[rl] = r < w.rows ? (uint32_t)(i * p.L + l) << 16 |
                                            (uint32_t)(w.kv * p.R + lr - l * p.R)
                                      : kNoRow;
            }
            row_tile_sync(wg);
            // q' of this row tile.  The last piece's MMAs are done (o_done), and
            // its O has been read: the MMAs of this piece wait for q_ready.
            {
                constexpr int LPR = D / 8;           // lanes a row, 8 values each
                constexpr int RPW = 32 / LPR;        // rows a warp at a time
                const int c = lane % LPR;
#pragma unroll 4  // loads under way together
                for (int r = (warp & 7) * RPW + lane / LPR; r < 128; r += 8 * RPW) {
                    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t id = rows[r];
                    if (id != kNoRow)
                        raw = *reinterpret_cast<const uint4 *>(
                            static_cast<const uint16_t *>(p.q) +
                            ((int64_t)w.b0 * p.L + (id >> 16)) * p.q_stride +
                            (int)(id & 0xffffu) * D + 8 * c);
                    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
                    float f[8], mx = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        f[i] = q_float(p, (uint16_t)(u[i / 2] >> (16 * (i & 1))));
                        mx = fmaxf(mx, fabsf(f[i]));
                    }
#pragma unroll
                    for (int o = LPR / 2; o >= 1; o >>= 1)
                        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
                    const int e = batch_exp(mx);
                    // a negative scale goes into q', so that the largest score
                    // is the largest of the products
                    const float sc = p.scale2 < 0.f ? -batch_pow2(e) : batch_pow2(e);
                    uint32_t h[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int a = BITS == 4 ? i : 2 * i, b = BITS == 4 ? i + 4 : 2 * i + 1;
                        h[i] = pack_half2(f[a] * sc, f[b] * sc);
                    }
                    *reinterpret_cast<uint4 *>(qs + wg * S::kQBytes + operand_at(128, r, c)) =
                        make_uint4(h[0], h[1], h[2], h[3]);
                    // never 0, which would make NaN of a masked score's -inf: products
                    // stay below 2^41, so the least normal factor scores 0 as well
                    if (c == 0)
                        qsc[wg * 128 + r] = fmaxf(batch_pow2(-e) * fabsf(p.scale2), FLT_MIN);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                row_tile_sync(wg);  // qsc of the row tile
                if (lane == 0) mbar_arrive(q_ready);
            }
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t o_at = tmem + lanes + S::kTmemO + wg * D + half * (D / 2);
            float *other = xch + (wg * 2 + (half ^ 1)) * 128 + rl;   // of the row's other half
            float *mine = xch + (wg * 2 + half) * 128 + rl;
            const float c = qsc[r];
            float m = 0.f;                  // reference of this row's weights
            float2 sum = make_float2(0.f, 0.f);
            for (int j = 0; j < tiles; ++j) {
                const uint32_t st = step + (row_tiles == 2 ? 2 * j + wg : j);
                const uint32_t slot = st & 1, s_at = tmem + lanes + slot * KT + half * KH;
                ok = ok && shd_wait(&s_full[slot], (st >> 1) & 1, p.err);
                tc_fence_after();
                // keys of this half that count
                const int valid = w.k1 - w.k0 - j * KT - half * KH;
                auto scores = [&](int k, uint32_t (&x)[32]) {
                    tmem_ld32(s_at + k, x);
                    tmem_wait_ld32(x);
                    if (k + 32 > valid) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (k + i >= valid) x[i] = 0xff800000u;  // -inf
                    }
                };
                // the row's largest score: of this half, then of both (two places
                // in turn, so that one barrier a tile is enough)
                float mx = -INFINITY;
#pragma unroll 1
                for (int k = 0; k < KH; k += 32) {
                    uint32_t x[32];
                    scores(k, x);
                    float a = mx, b = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        a = fmaxf(a, fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 1])));
                        b = fmaxf(b, fmaxf(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])));
                    }
                    mx = fmaxf(a, b);
                }
                const int turn = (j & 1) * S::kRT * 256;
                mine[turn] = mx;
                ok = row_tile_all(wg, ok);
                if (!ok) break;
                mx = fmaxf(mx, other[turn]) * c;
                // the reference moves when a weight could pass 2^15
                float f = 1.f;
                if (j == 0) {
                    m = mx == -INFINITY ? 0.f : mx;
                } else if (mx > m + kMove) {
                    f = batch_ex2(m - mx);
                    m = mx;
                }
                if (__any_sync(~0u, f != 1.f)) {
                    // O of the tiles so far, once their products are done
                    // (with two row tiles these scores follow the last one)
                    const uint32_t n = kt + j - 1;
                    if (row_tiles == 1)  // (one that gives up is told of at the next barrier)
                        ok = shd_wait(&v_empty[n & 1], (n >> 1) & 1, p.err);
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < D / 2; k += 8) {
                        uint32_t o[8];
                        tmem_ld8(o_at + k, o);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st8(o_at + k, o);
                    }
                    sum.x *= f;
                    sum.y *= f;
                }
                const float2 c2 = make_float2(c, c), m2 = make_float2(kRoom - m, kRoom - m);
                // P of scores k .. k + 31 takes 16 columns at k / 2 of this half's,
                // over scores that have been read
                float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll 1
                for (int k = 0; k < KH; k += 32) {
                    uint32_t x[32], h[16];
                    scores(k, x);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 t = __ffma2_rn(make_float2(__uint_as_float(x[2 * i]),
                                                          __uint_as_float(x[2 * i + 1])),
                                              c2, m2);
                        t.x = batch_ex2(t.x);
                        t.y = batch_ex2(t.y);
                        if (i & 1)
                            sum = __fadd2_rn(sum, t);
                        else
                            sum2 = __fadd2_rn(sum2, t);
                        h[i] = pack_half2(t.x, t.y);
                    }
                    tmem_st16(s_at + k / 2, h);
                }
                sum = __fadd2_rn(sum, sum2);
                tmem_wait_st();
                tc_fence_before();
                ok = __all_sync(~0u, ok);
                if (lane == 0 && ok) mbar_arrive(&p_ready[slot]);
            }
            // ----------------------------------------------------- partial out
            if (ok) ok = shd_wait(o_done, piece & 1, p.err);
            ok = row_tile_all(wg, ok);  // (and the last tile's exchange has been read)
            *mine = sum.x + sum.y;
            row_tile_sync(wg);
            if (ok) {
                tc_fence_after();
                auto part = [&](uint32_t id) {
                    return ((int64_t)w.slot0 * p.L + (id >> 16)) * p.H + (id & 0xffffu);
                };
                if (half == 0 && rows[rl] != kNoRow)
                    p.part_ml[part(rows[rl])] = make_float2(m - kRoom, *mine + *other);
                // O through this row tile's q' (done with), a quarter of the columns
                // at a time: a thread has a row, but memory wants a row's columns
                // next to each other.  Chunks of 16 bytes, swizzled by row.
                constexpr int CR = D / 4, CH = CR / 4;
                float4 *stage = reinterpret_cast<float4 *>(qs + wg * S::kQBytes + half * (S::kQBytes / 2)) +
                                (warp & 3) * 32 * CH;
                auto spot = [&](int row, int chunk) {
                    return row * CH + (chunk ^ (D == 64 ? (row >> 1) & 3 : row & 7));
                };
#pragma unroll 1
                for (int round = 0; round < 2; ++round) {
#pragma unroll
                    for (int k = 0; k < CR; k += 16) {
                        uint32_t u[16];
                        tmem_ld16w(o_at + round * CR + k, u);
                        constexpr int i1 = BITS == 4 ? 2 : 1, i4 = BITS == 4 ? 1 : 4;
#pragma unroll
                        for (int g = 0; g < 16; g += 8) {
                            const uint32_t *x = u + g;
                            stage[spot(lane, (k + g) / 4)] = make_float4(
                                __uint_as_float(x[0]), __uint_as_float(x[i1]),
                                __uint_as_float(x[2 * i1]), __uint_as_float(x[3 * i1]));
                            stage[spot(lane, (k + g) / 4 + 1)] = make_float4(
                                __uint_as_float(x[i4]), __uint_as_float(x[i4 + i1]),
                                __uint_as_float(x[i4 + 2 * i1]), __uint_as_float(x[i4 + 3 * i1]));
                        }
                    }
                    __syncwarp();
#pragma unroll 4
                    for (int i = lane; i < 32 * CH; i += 32) {
                        const int row = i / CH, chunk = i % CH;
                        const uint32_t id = rows[(warp & 3) * 32 + row];
                        if (id != kNoRow)
                            reinterpret_cast<float4 *>(p.part_o + part(id) * D + half * (D / 2) +
                                                       round * CR)[chunk] = stage[spot(row, chunk)];
                    }
                    __syncwarp();
                }
            }
            row_tile_sync(wg);  // the exchange is read before the next piece's
            tc_fence_before();
            kt += tiles;
            step += tiles * row_tiles;
        }
    } else if (warp < 24) {
        // -------------------------------------------------------- dequantise
        for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
            const Piece w = shared_piece(p, item);
            const int tiles = (w.k1 - w.k0 + KT - 1) / KT;
            // A warp takes KT / 8 consecutive keys (within one page) of every
            // tile: 16 bytes of codes a lane, kLpr lanes a row, so that a
            // load covers 512 bytes in a row.
            const int dw = warp - 16;
            const int key0 = dw * S::kWKeys, row = lane / S::kLpr, l = lane % S::kLpr;
            const int32_t *trow = p.table + (int64_t)w.row * p.max_pages;
            struct Raw {
                uint4 c[S::kLoads];
                __half2 sb[S::kLoads];
            };
            // (Tables and pages are read by ordinary loads: this grid may have started
            // while an earlier one still wrote them, so they are not constant.)
            // the record of this warp's keys of tile j; nullptr past the end,
            // or where the table names no page of the pool
            auto place = [&](int j) -> const uint8_t * {
                const int at = w.k0 + j * KT + key0;
                if (j >= tiles || at >= w.k1) return nullptr;
                const int id = trow[at >> p.c.page_log2];
                if (id < 0 || id >= p.c.n_pages) {
                    if (lane == 0) atomicOr(p.err, ERR_BATCH_TABLE);
                    return nullptr;
                }
                return p.layer + id * p.c.page_bytes + w.kv * p.c.rec;
            };
            auto fetch = [&](Raw &x, const uint8_t *rec, int j, int which) {
                const int at = w.k0 + j * KT + key0, slot = at & (p.c.page - 1);
                const uint4 *c = reinterpret_cast<const uint4 *>(
                                     rec + which * p.c.side_codes + slot * S::kRB) + lane;
                const __half2 *sb = reinterpret_cast<const __half2 *>(
                                        rec + 2 * (int64_t)p.c.side_codes + which * p.c.side_sb) +
                                    (slot + row) * S::kG + l * S::kLane / GROUP;
#pragma unroll
                for (int i = 0; i < S::kLoads; ++i) {
                    const bool in = rec && at + row + i * S::kLRows < w.k1;
                    x.c[i] = in ? __ldca(c + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
                    x.sb[i] = in ? __ldca(sb + i * S::kLRows * S::kG) : __float2half2_rn(0.f);
                }
            };
            // the lines of the tile after the next into L2
            auto prefetch = [&](const uint8_t *rec, int j) {
                if (!rec) return;
                const int slot = (w.k0 + j * KT + key0) & (p.c.page - 1);
                constexpr int kLines = (S::kWKeys * S::kRB + 127) / 128;  // of K codes, of V codes
                for (int i = lane; i < 2 * kLines; i += 32)
                    prefetch_l2(rec + (i < kLines ? 0 : p.c.side_codes) + slot * S::kRB +
                                128 * (i < kLines ? i : i - kLines));
                if (lane < 2)
                    prefetch_l2(rec + 2 * (int64_t)p.c.side_codes + lane * p.c.side_sb +
                                slot * S::kG * 4);
            };
            const int turn = BITS == 4 ? (l >> 1) * (D == 128 ? 2 : 1) & 3 : (l >> 2) & 1;
            // whether values of x could pass the largest fp16 number (pairs that
            // are not finite leave theirs as they are)
            auto past = [&](const Raw &x) {
                __half2 most = __habs2(x.sb[0]);
#pragma unroll
                for (int i = 1; i < S::kLoads; ++i) most = __hmax2_nan(most, __habs2(x.sb[i]));
                return past_fp16<BITS>(most) && __hble2(most, __float2half2_rn(65504.f));
            };
            auto store = [&](const Raw &x, uint8_t *tile, bool past) {
#pragma unroll
                for (int i = 0; i < S::kLoads; ++i) {
                    const __half2 s = __low2half2(x.sb[i]), b = __high2half2(x.sb[i]);
                    // the lane's 16-byte chunks are stored in an order turned by
                    // lane, so that 8 lanes store to 8 distinct bank groups;
                    // swaps bring the words of chunk k ^ turn to place k
                    uint32_t cw[4] = {x.c[i].x, x.c[i].y, x.c[i].z, x.c[i].w};
                    auto swap = [&](bool on, int u, int v) {
                        const uint32_t t = on ? cw[v] : cw[u];
                        cw[v] = on ? cw[u] : cw[v];
                        cw[u] = t;
                    };
                    if constexpr (BITS == 4) {
                        swap(turn & 1, 0, 1);
                        swap(turn & 1, 2, 3);
                        swap(turn & 2, 0, 2);
                        swap(turn & 2, 1, 3);
                    } else {
                        swap(turn & 1, 0, 2);
                        swap(turn & 1, 1, 3);
                    }
                    const uint32_t at =
                        operand_at(KT, key0 + row + i * S::kLRows, l * S::kChunks) ^
                        ((uint32_t)turn << 4);
#pragma unroll
                    for (int k = 0; k < S::kChunks; ++k)
                        *reinterpret_cast<uint4 *>(tile + (at ^ ((uint32_t)k << 4))) =
                            values8<BITS>(cw + k * BITS / 4, s, b);
                }
                if (__builtin_expect(past, 0)) clip_fp16<S>(smem_u32(tile), key0 + row, l);
                fence_proxy_async_smem();
                __syncwarp();
            };
            // k and v of a tile in turn, by the same code; the next codes are
            // under way while these are turned into values
            Raw x, y;
            const uint8_t *rec = place(0), *rec1 = place(1);
            fetch(x, rec, 0, 0);
            prefetch(rec1, 1);
#pragma unroll 1
            for (int h = 0; h < 2 * tiles; ++h) {
                const int j = h >> 1, which = h & 1;
                const uint32_t n = kt + j, s = n & 1, lap = n >> 1;
                fetch(y, which ? rec1 : rec, j + which, which ^ 1);
                if (which) {
                    rec = rec1;
                    rec1 = place(j + 2);
                    prefetch(rec1, j + 2);
                }
                uint64_t *empty = which ? &v_empty[s] : row_tiles == 1 ? &s_full[s] : &k_empty[s];
                const bool top = past(x);
                const bool ok =
                    lap == 0 || shd_wait(empty, (lap - 1) & 1, p.err);
                if (!__all_sync(~0u, ok)) goto wound_down;
                store(x, (which ? vs : ks) + s * S::kTileBytes, top);
                const bool withheld = p.withhold && n == 0 && !which;  // tests: nothing completes k_full[0]
                if (lane == 0 && !withheld) mbar_arrive(which ? &v_full[s] : &k_full[s]);
                x = y;
            }
            kt += tiles;
        }
    } else {
        // --------------------------------------------------------------- MMA
        // One thread waits and issues.  A step's value product and the scores
        // two steps on go out together, then the commits.  Its time is its own
        // instructions (the roles' code crowds the instruction caches, and a
        // wait costs 150 cycles even when it is over): no wait twice, offsets
        // known when compiled.
        if (elect_lane()) {
            const uint32_t id_s =
                (1u << 4) | ((uint32_t)(KT >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
            const uint32_t id_o = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) |
                                  ((uint32_t)(128 >> 4) << 24);
            const uint64_t qd = sw128_desc(smem_u32(qs)), kd0 = sw128_desc(smem_u32(ks));
            const uint64_t vd0 = mn_desc(smem_u32(vs), KT * 128);
            // scores of row tile t with the k tile in slot s, to score slot `to`
            auto scores = [&](int t, uint32_t s, uint32_t to) {
                const uint64_t a = qd + (uint64_t)((t * S::kQBytes) >> 4);
                const uint64_t b = kd0 + (s ? (uint64_t)(S::kTileBytes >> 4) : 0);
                const uint32_t d = tmem + to * KT;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc_mma_f16(d, a + (uint64_t)(((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                               b + (uint64_t)(((k >> 2) * (KT * 128) + (k & 3) * 32) >> 4), id_s,
                               k != 0);
            };
            // O of row tile t (+)= P in score slot `from` x the v tile in slot s
            auto values = [&](int t, uint32_t s, uint32_t from, uint32_t more) {
                const uint32_t a = tmem + from * KT, d = tmem + S::kTmemO + t * D;
                const uint64_t b = vd0 + (s ? (uint64_t)(S::kTileBytes >> 4) : 0);
#pragma unroll
                for (int k = 0; k < KT / 16; ++k)
                    tc_mma_f16_ta(d, a + (k / (KT / 32)) * (KT / 2) + (k % (KT / 32)) * 8,
                                  b + (uint64_t)((k * 2048) >> 4), id_o, k != 0 ? 1u : more);
            };
            auto wait = [&](uint64_t *bar, uint32_t n) {
                return shd_wait(bar, n & 1, p.err);
            };
            bool ok = true;
            for (int item = blockIdx.x; ok && item < n_items; item += gridDim.x, ++piece) {
                const Piece w = shared_piece(p, item);
                const int tiles = (w.k1 - w.k0 + KT - 1) / KT;
                ok = wait(q_ready, piece) && wait(&k_full[kt & 1], kt >> 1);
                if (!ok) break;
                tc_fence_after();
                issued = true;
                if (row_tiles == 2) {
                    // score slot = row tile; both row tiles use each k and v tile
                    scores(0, kt & 1, 0);
                    tc_commit(&s_full[0]);
                    scores(1, kt & 1, 1);
                    tc_commit(&s_full[1]);
                    tc_commit(&k_empty[kt & 1]);
                    ok = wait(&v_full[kt & 1], kt >> 1);
#pragma unroll 1
                    for (int j = 0; ok && j < tiles; ++j, ++kt) {
                        const uint32_t s = kt & 1, n = kt + 1;
                        const bool next = j + 1 < tiles;
                        ok = (!next || wait(&k_full[n & 1], n >> 1)) && wait(&p_ready[0], kt);
                        if (!ok) break;
                        tc_fence_after();
                        values(0, s, 0, j != 0);
                        if (next) {
                            scores(0, n & 1, 0);
                            tc_commit(&s_full[0]);
                            // in the time until P of the other row tile
                            ok = wait(&v_full[n & 1], n >> 1);
                        }
                        ok = ok && wait(&p_ready[1], kt);
                        if (!ok) break;
                        tc_fence_after();
                        values(1, s, 1, j != 0);
                        if (next) {
                            scores(1, n & 1, 1);
                            tc_commit(&s_full[1]);
                            tc_commit(&k_empty[n & 1]);
                        }
                        tc_commit(&v_empty[s]);
                    }
                    if (!ok) break;
                } else {
                    // score slot = k and v slot; s_full also says that k is free
                    scores(0, kt & 1, kt & 1);
                    tc_commit(&s_full[kt & 1]);
                    if (tiles > 1) {
                        ok = wait(&k_full[(kt + 1) & 1], (kt + 1) >> 1);
                        if (!ok) break;
                        tc_fence_after();
                        scores(0, (kt + 1) & 1, (kt + 1) & 1);
                        tc_commit(&s_full[(kt + 1) & 1]);
                    }
#pragma unroll 1
                    for (int j = 0; j < tiles; ++j, ++kt) {
                        const uint32_t s = kt & 1;
                        const bool next = j + 2 < tiles;
                        ok = wait(&v_full[s], kt >> 1) && (!next || wait(&k_full[s], (kt + 2) >> 1)) &&
                             wait(&p_ready[s], kt >> 1);
                        if (!ok) break;
                        tc_fence_after();
                        values(0, s, s, j != 0);
                        if (next) {
                            scores(0, s, s);
                            tc_commit(&s_full[s]);
                        }
                        tc_commit(&v_empty[s]);
                    }
                }
                tc_commit(o_done);
            }
        }
        __syncwarp();
    }
wound_down:
    // every MMA that was issued has completed before tensor memory is freed
    if (issued) {  // the issuing thread
        tc_commit(drain);
        if (!mbar_wait(drain, 0)) atomicOr(p.err, ERR_BATCH_BASE);
    }
    __syncthreads();
    if (warp == 24) tmem_dealloc(tmem, 512);
}

template <int BITS, int D, int GROUP>
cudaError_t shared_run(const BatchParams &p, int row_tiles, int grid, cudaStream_t stream) {
    using S = Shd<BITS, D, GROUP>;
    auto kern = shared_kernel<BITS, D, GROUP>;
    constexpr size_t body = 1024 + (size_t)S::kRT * S::kQBytes + 4 * (size_t)S::kTileBytes +
                            S::kRT * 3072 + 18 * 8;
    static std::once_flag once;
    static cudaError_t attr = cudaSuccess;
    std::call_once(once, [&] {
        attr = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)body);
    });
    if (attr != cudaSuccess) return attr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(S::kThreads, 1, 1);
    cfg.dynamicSmemBytes = body;
    cfg.stream = stream;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = a;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p, row_tiles);
}

template <int BITS, int D>
cudaError_t shared_group(const BatchParams &p, int row_tiles, int grid, cudaStream_t stream) {
    if (p.c.group == 32) return shared_run<BITS, D, 32>(p, row_tiles, grid, stream);
    if (p.c.group == 64) return shared_run<BITS, D, 64>(p, row_tiles, grid, stream);
    if constexpr (D >= 128) return shared_run<BITS, D, 128>(p, row_tiles, grid, stream);
    return cudaErrorInvalidValue;
}

template <int BITS>
cudaError_t shared_dim(const BatchParams &p, int row_tiles, int grid, cudaStream_t stream) {
    switch (p.c.D) {
        case 64: return shared_group<BITS, 64>(p, row_tiles, grid, stream);
        case 128: return shared_group<BITS, 128>(p, row_tiles, grid, stream);
        case 256: return shared_group<BITS, 256>(p, row_tiles, grid, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t batch_shared(const BatchParams &p, int row_tiles, int grid, cudaStream_t stream) {
    return p.c.bits == 4 ? shared_dim<4>(p, row_tiles, grid, stream)
                         : shared_dim<8>(p, row_tiles, grid, stream);
}

}  // namespace aq
