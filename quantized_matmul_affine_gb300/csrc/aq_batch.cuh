// Attention of a batch over the paged quantised cache: parameters and the
// plan that its kernels share.
//
// The work of a call is cut into pieces of keys: the shared keys of a group
// (read once for all the group's rows) and each sequence's own keys.  A piece
// leaves, for every row (token, head) it serves, a partial result in a slot of
// the workspace: the largest score (in log2 units), the sum of weights and
// the unnormalised output, fp32.  The slots of a row are added in a fixed
// order afterwards.  All lengths are known to the device only, so every CTA
// works out the same plan from lens, group_start and shared by itself.
#pragma once

#include "aq_cache.cuh"
#include "aq_ptx.cuh"

namespace aq {

constexpr int kBatchMaxGroups = AQ_BATCH_MAX_GROUPS;

struct BatchParams {
    CacheGeom c;
    const uint8_t *layer;    // the layer's pages
    const void *q;
    void *out;
    int64_t q_stride;
    const int32_t *table, *lens, *gstart, *shared;
    int64_t max_pages;
    int B, L, H, R, G;       // R = H / KV query heads a KV head
    int bf16;
    float scale2;            // scale * log2(e)
    float *part_o;           // [slots][L][H][D]
    float2 *part_ml;         // [slots][L][H]
    int32_t *desc;           // [B][5], see PlanView
    int64_t slots;           // slots of the workspace
    int64_t key_cap;         // max_pages * page, at most 2^29
    int own_target;          // pieces x KV heads x row tiles wanted of own keys
    int own_rows;            // rows a tile of the kernel for own keys
    int shared_target;       // the same of shared keys
    int shared_rows;
    int shared_unit;         // piece lengths are multiples of these
    int own_unit;
    uint32_t *err;
};

// What a CTA knows after batch_plan, in shared memory.
struct PlanView {
    int *start;    // [B] first own key
    int *sbase;    // [B + 1] own pieces before row b
    int *gidx;     // [B] group that row b shares with, or -1
    int *g_len;    // [G] shared keys (0: nobody shares)
    int *g_lead;   // [G] row whose table entries serve them
    int *g_items;  // [G + 1] (piece, row tile) pairs before group g
    int *g_slot;   // [G] first slot
    int *g_first;  // [G] first row
    int *g_rows;   // [G] rows of the group
    int own_chunk, shared_chunk;
    int own_items, shared_items;  // pieces (x row tiles for shared), per KV head
    int shared_slots;
};

__host__ __device__ inline size_t plan_bytes(int B, int G) {
    return sizeof(int) * ((size_t)3 * B + 1 + (size_t)6 * G + 1 + 64);
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (int)(((int64_t)a + b - 1) / b); }

// Sum over the CTA, returned to every thread; tmp: 33 ints.
__device__ __forceinline__ int64_t block_sum(int64_t v, long long *tmp) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if (lane == 0) tmp[warp] = v;
    __syncthreads();
    int64_t s = 0;
    for (int w = 0; w < nw; ++w) s += tmp[w];
    __syncthreads();  // tmp may be written again
    return s;
}

// Own pieces of row b for pieces of `chunk` keys.
__device__ __forceinline__ int own_pieces(const BatchParams &p, const PlanView &v, int b,
                                          int chunk) {
    const int n = min((int)p.key_cap, max(0, __ldg(p.lens + b))) - v.start[b];
    return n > 0 ? ceil_div(n, chunk) : 0;
}

// The plan, by all threads of a CTA (a multiple of 32, at most 1024).  mem:
// plan_bytes(B, G); tmp: 33 long longs.
__device__ inline PlanView batch_plan(const BatchParams &p, int *mem, long long *tmp) {
    PlanView v;
    v.start = mem;
    v.sbase = v.start + p.B;
    v.gidx = v.sbase + p.B + 1;
    v.g_len = v.gidx + p.B;
    v.g_lead = v.g_len + p.G;
    v.g_items = v.g_lead + p.G;
    v.g_slot = v.g_items + p.G + 1;
    v.g_first = v.g_slot + p.G;
    v.g_rows = v.g_first + p.G;
    int *g_count = v.g_items;  // until the items are counted
    const int nt = blockDim.x, cap = (int)p.key_cap;
    int disorder = 0;
    for (int g = threadIdx.x; g < p.G; g += nt) {
        const int b0 = __ldg(p.gstart + g), b1 = __ldg(p.gstart + g + 1);
        disorder |= b0 < 0 || b1 < b0 || b1 > p.B;
        v.g_first[g] = b0;
        v.g_rows[g] = b1 - b0;
        v.g_len[g] = min(cap, max(0, __ldg(p.shared + g)));
        v.g_lead[g] = p.B;
        g_count[g] = 0;
    }
    // groups that do not ascend within the batch share nothing
    if (p.G > 0 && __syncthreads_or(disorder)) {
        for (int g = threadIdx.x; g < p.G; g += nt) v.g_first[g] = v.g_rows[g] = v.g_len[g] = 0;
        if (threadIdx.x == 0) atomicOr(p.err, ERR_BATCH_TABLE);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += nt) {
        int g = -1;
        if (p.G > 0) {
            int lo = 0, hi = p.G;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (v.g_first[mid] <= b)
                    lo = mid;
                else
                    hi = mid;
            }
            const int len = min(cap, __ldg(p.lens + b));
            if (b >= v.g_first[lo] && b < v.g_first[lo] + v.g_rows[lo] && v.g_len[lo] > 0 &&
                len - (p.L - 1) >= v.g_len[lo]) {
                g = lo;
                atomicMin(&v.g_lead[lo], b);
                atomicAdd(&g_count[lo], 1);
            }
        }
        v.gidx[b] = g;
    }
    __syncthreads();
    // a group of one shares with nobody
    for (int g = threadIdx.x; g < p.G; g += nt)
        if (g_count[g] < 2) v.g_len[g] = 0;
    __syncthreads();
    int64_t own = 0;
    for (int b = threadIdx.x; b < p.B; b += nt) {
        int g = v.gidx[b];
        if (g >= 0 && v.g_len[g] == 0) v.gidx[b] = g = -1;
        v.start[b] = g >= 0 ? v.g_len[g] : 0;
        own += max(0, min(cap, __ldg(p.lens + b)) - v.start[b]);
    }
    // units of work: keys x row tiles x KV heads
    const int own_tiles = ceil_div(p.L * p.R, p.own_rows);
    own = block_sum(own, tmp) * own_tiles * p.c.KV;
    int64_t sh = 0;
    for (int g = threadIdx.x; g < p.G; g += nt)
        sh += (int64_t)v.g_len[g] * ceil_div(v.g_rows[g] * p.L * p.R, p.shared_rows) * p.c.KV;
    sh = block_sum(sh, tmp);
    auto piece = [](int64_t units, int target, int unit) {
        const int64_t each = (units + target - 1) / target;
        return (int)min((int64_t)(1 << 29), max((int64_t)unit, (each + unit - 1) / unit * unit));
    };
    v.own_chunk = piece(own, p.own_target, p.own_unit);
    v.shared_chunk = piece(sh, p.shared_target, p.shared_unit);
    // one piece more than the device holds at once would cost a whole round:
    // shared pieces grow until they fit (each group has at least one)
    for (int k = 0; k < 8 && p.G > 0; ++k) {
        int64_t n = 0;
        for (int g = threadIdx.x; g < p.G; g += nt)
            n += (int64_t)ceil_div(v.g_len[g], v.shared_chunk) *
                 ceil_div(v.g_rows[g] * p.L * p.R, p.shared_rows) * p.c.KV;
        n = block_sum(n, tmp);
        if (n <= p.shared_target || v.shared_chunk >= cap) break;
        const int64_t want = ((int64_t)v.shared_chunk * n / p.shared_target + p.shared_unit - 1) /
                             p.shared_unit * p.shared_unit;
        v.shared_chunk = (int)min((int64_t)(1 << 29), max(want, (int64_t)v.shared_chunk + p.shared_unit));
    }
    // pieces grow until their slots fit the workspace
    for (;;) {
        int64_t n = 0;
        for (int b = threadIdx.x; b < p.B; b += nt) n += own_pieces(p, v, b, v.own_chunk);
        for (int g = threadIdx.x; g < p.G; g += nt)
            n += (int64_t)ceil_div(v.g_len[g], v.shared_chunk) * v.g_rows[g];
        if (block_sum(n, tmp) <= p.slots || (v.own_chunk >= cap && v.shared_chunk >= cap)) break;
        if (v.own_chunk < cap) v.own_chunk *= 2;
        if (v.shared_chunk < cap) v.shared_chunk *= 2;
    }
    // groups' items and slots (warp 0), then the rows' pieces
    if (threadIdx.x < 32) {
        int items = 0, slots = 0;
        for (int g0 = 0; g0 < p.G; g0 += 32) {
            const int g = g0 + threadIdx.x;
            int it = 0, sl = 0;
            if (g < p.G) {
                const int n = ceil_div(v.g_len[g], v.shared_chunk);
                it = n * ceil_div(v.g_rows[g] * p.L * p.R, p.shared_rows);
                sl = n * v.g_rows[g];
            }
            int bi = it, bs = sl;
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(~0u, bi, o), y = __shfl_up_sync(~0u, bs, o);
                if ((int)threadIdx.x >= o) bi += x, bs += y;
            }
            if (g < p.G) {
                v.g_items[g] = items + bi - it;
                v.g_slot[g] = slots + bs - sl;
            }
            items += __shfl_sync(~0u, bi, 31);
            slots += __shfl_sync(~0u, bs, 31);
        }
        if (threadIdx.x == 0) {
            v.g_items[p.G] = items;
            tmp[0] = items;
            tmp[1] = slots;
        }
    }
    __syncthreads();
    v.shared_items = (int)tmp[0];
    v.shared_slots = (int)tmp[1];
    __syncthreads();
    int carry = 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int b0 = 0; b0 < p.B; b0 += nt) {
        const int b = b0 + threadIdx.x;
        const int n = b < p.B ? own_pieces(p, v, b, v.own_chunk) : 0;
        int before = n;
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(~0u, before, o);
            if (lane >= o) before += x;
        }
        if (lane == 31) tmp[warp] = before;
        __syncthreads();
        int skip = carry, all = carry;
        for (int w = 0; w < nt >> 5; ++w) {
            if (w < warp) skip += (int)tmp[w];
            all += (int)tmp[w];
        }
        carry = all;
        if (b < p.B) v.sbase[b] = skip + before - n;
        __syncthreads();
    }
    if (threadIdx.x == 0) v.sbase[p.B] = carry;
    v.own_items = carry;
    __syncthreads();
    return v;
}

// For the kernel that adds the slots: per row b its first own slot, own
// pieces, first shared slot, step from one shared piece to the next, pieces.
__device__ inline void write_desc(const BatchParams &p, const PlanView &v) {
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
        const int g = v.gidx[b];
        int32_t *d = p.desc + 5 * b;
        d[0] = v.shared_slots + v.sbase[b];
        d[1] = v.sbase[b + 1] - v.sbase[b];
        d[2] = g >= 0 ? v.g_slot[g] + (b - v.g_first[g]) : 0;
        d[3] = g >= 0 ? v.g_rows[g] : 0;
        d[4] = g >= 0 ? ceil_div(v.g_len[g], v.shared_chunk) : 0;
    }
}

// The last index i in [0, n) with base[i] <= x (base ascends, base[0] <= x).
__device__ __forceinline__ int last_at_most(const int *base, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (base[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// A piece of work of one CTA: keys [k0, k1) of table row `row`, for the rows
// [r0, r0 + n) of sequences from b0 on (row r: sequence b0 + r / (L * R),
// token r / R % L, query head r % R of KV head kv), partial results to slot
// slot0 + r / (L * R).
struct Piece {
    int row, k0, k1, b0, r0, rows, kv, slot0;
};

// The i-th piece of the shared keys, i < shared_items * KV: row tiles
// fastest, so that the tiles that read the same keys run together.
__device__ __forceinline__ Piece shared_piece(const BatchParams &p, const PlanView &v, int i,
                                              int tile_rows) {
    Piece w;
    // item = ((piece * KV) + kv) * tiles + tile within the group
    const int KV = p.c.KV;
    int lo = 0, hi = p.G;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)v.g_items[mid] * KV <= i)
            lo = mid;
        else
            hi = mid;
    }
    // groups without items have their successor's base: lo is the last
    const int g = lo, rows = v.g_rows[g] * p.L * p.R, tiles = ceil_div(rows, tile_rows);
    const int rem = i - v.g_items[g] * KV;
    const int tile = rem % tiles, kc = rem / tiles, kv = kc % KV, chunk = kc / KV;
    w.row = v.g_lead[g];
    w.k0 = chunk * v.shared_chunk;
    w.k1 = min(v.g_len[g], w.k0 + v.shared_chunk);
    w.b0 = v.g_first[g];
    w.r0 = tile * tile_rows;
    w.rows = min(tile_rows, rows - w.r0);
    w.kv = kv;
    w.slot0 = v.g_slot[g] + chunk * v.g_rows[g];
    return w;
}

__device__ __forceinline__ Piece own_piece(const BatchParams &p, const PlanView &v, int i,
                                           int tile_rows) {
    Piece w;
    const int tiles = ceil_div(p.L * p.R, tile_rows);
    const int tile = i % tiles, kc = i / tiles, kv = kc % p.c.KV, q = kc / p.c.KV;
    const int b = last_at_most(v.sbase, p.B, q);
    const int chunk = q - v.sbase[b];
    w.row = w.b0 = b;
    w.k0 = v.start[b] + chunk * v.own_chunk;
    w.k1 = min(min((int)p.key_cap, __ldg(p.lens + b)), w.k0 + v.own_chunk);
    w.r0 = tile * tile_rows;
    w.rows = min(tile_rows, p.L * p.R - w.r0);
    w.kv = kv;
    w.slot0 = v.shared_slots + q;
    return w;
}

__device__ __forceinline__ float batch_pow2(int e) { return __int_as_float((127 + e) << 23); }

// v * 2^result lies in [2^14, 2^15); clamped so that every power used is a
// normal float.
__device__ __forceinline__ int batch_exp(float v) {
    const int ex = (int)(__float_as_uint(v) >> 23 & 255u) - 126;
    return v > 0.f ? max(-100, min(100, 15 - ex)) : 100;
}

__device__ __forceinline__ float batch_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// q of one row (piece w, row r of its tile), 4-byte pairs: element pointer.
__device__ __forceinline__ const uint16_t *q_row(const BatchParams &p, const Piece &w, int r) {
    const int LR = p.L * p.R, i = (w.r0 + r) / LR, lr = (w.r0 + r) - i * LR;
    const int l = lr / p.R, h = w.kv * p.R + (lr - l * p.R);
    return static_cast<const uint16_t *>(p.q) +
           ((int64_t)(w.b0 + i) * p.L + l) * p.q_stride + (int64_t)h * p.c.D;
}
// Index of the row's partial result: ((slot * L) + l) * H + h.
__device__ __forceinline__ int64_t part_row(const BatchParams &p, const Piece &w, int r) {
    const int LR = p.L * p.R, i = (w.r0 + r) / LR, lr = (w.r0 + r) - i * LR;
    const int l = lr / p.R, h = w.kv * p.R + (lr - l * p.R);
    return ((int64_t)(w.slot0 + i) * p.L + l) * p.H + h;
}
__device__ __forceinline__ float q_float(const BatchParams &p, uint16_t v) {
    return p.bf16 ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
}

}  // namespace aq
