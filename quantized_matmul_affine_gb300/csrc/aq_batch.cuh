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
//
// Two kernels take pieces.  shared_kernel (tensor core, many rows) takes
// ranges of shared_chunk keys of a group.  own_kernel takes own keys, and
// shared keys of groups of few rows: its tiles of unit_keys keys, in order of
// (group or sequence, KV head, row tile, key), are dealt to its warps in even
// runs of `per` tiles, so that all warps have the same work however uneven
// the sequences are.
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
    int32_t *desc;           // see write_desc
    int64_t slots;           // slots of the workspace
    int64_t key_cap;         // max_pages * page, at most 2^29
    int own_rows;            // query rows a tile of own_kernel
    int own_warps;           // its warps
    int own_min;             // tiles a warp takes at least
    int unit_keys;           // keys a tile
    int shared_tc;           // shared_kernel takes the shared keys (else own_kernel)
    int shared_target;       // its CTAs
    int shared_rows;         // query rows a tile of it
    int shared_unit;         // its chunks are multiples of this
    uint32_t *err;
};

// What a CTA knows after batch_plan, in shared memory.
struct PlanView {
    int64_t *ubase;    // [B + 1] tiles of own_kernel before row b's own keys
    int64_t *g_ubase;  // [G + 1] the same before group g's (groups come first)
    int *start;        // [B] first own key
    int *sbase;        // [B] first slot of the own keys
    int *gidx;         // [B] group that row b shares with, or -1
    int *g_len;        // [G] shared keys (0: nobody shares)
    int *g_lead;       // [G] row whose table entries serve them
    int *g_items;      // [G + 1] shared_kernel's (chunk, row tile) pairs before group g
    int *g_slot;       // [G] first slot
    int *g_first;      // [G] first row
    int *g_rows;       // [G] rows of the group
    int64_t per;       // tiles a warp of own_kernel takes
    int shared_chunk;  // keys a chunk of shared_kernel
    int shared_items;  // g_items[G]
};

__host__ __device__ inline size_t plan_bytes(int B, int G) {
    return sizeof(int64_t) * ((size_t)B + G + 3) +
           sizeof(int) * ((size_t)3 * B + 6 * (size_t)G + 2);
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (int)(((int64_t)a + b - 1) / b); }

// Sum over the CTA, returned to every thread; tmp: 32 values.
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

// Sum over the CTA's threads before this one, and over all; tmp as above.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *total, long long *tmp) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    int64_t upto = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) tmp[warp] = upto;
    __syncthreads();
    int64_t skip = 0, all = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < warp) skip += tmp[w];
        all += tmp[w];
    }
    __syncthreads();
    *total = all;
    return skip + upto - v;
}

// Tiles of own_kernel that row b's own keys take.
__device__ __forceinline__ int own_tiles(const BatchParams &p, const PlanView &v, int b) {
    const int len = min((int)p.key_cap, __ldg(p.lens + b));
    return len > v.start[b] ? ceil_div(len, p.unit_keys) - v.start[b] / p.unit_keys : 0;
}
// Slots that a segment of so many tiles may need: the runs it can touch.
__device__ __forceinline__ int64_t seg_slots(int64_t tiles, int64_t per) {
    return tiles > 0 ? (tiles - 1) / per + 2 : 0;
}

// The plan, by all threads of a CTA (a multiple of 32, at most 1024).  mem:
// plan_bytes(B, G); tmp: 32 values.
__device__ inline PlanView batch_plan(const BatchParams &p, int *mem, long long *tmp) {
    PlanView v;
    v.ubase = reinterpret_cast<int64_t *>((reinterpret_cast<uintptr_t>(mem) + 7) & ~(uintptr_t)7);
    v.g_ubase = v.ubase + p.B + 1;
    v.start = reinterpret_cast<int *>(v.g_ubase + p.G + 1);
    v.sbase = v.start + p.B;
    v.gidx = v.sbase + p.B;
    v.g_len = v.gidx + p.B;
    v.g_lead = v.g_len + p.G;
    v.g_items = v.g_lead + p.G;
    v.g_slot = v.g_items + p.G + 1;
    v.g_first = v.g_slot + p.G;
    v.g_rows = v.g_first + p.G;
    int *g_count = v.g_items;  // until the items are counted
    const int nt = blockDim.x, cap = (int)p.key_cap;
    if (p.G > 0) {
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
        if (__syncthreads_or(disorder)) {
            for (int g = threadIdx.x; g < p.G; g += nt)
                v.g_first[g] = v.g_rows[g] = v.g_len[g] = 0;
            if (threadIdx.x == 0) atomicOr(p.err, ERR_BATCH_TABLE);
        }
        __syncthreads();
        for (int b = threadIdx.x; b < p.B; b += nt) {
            int lo = 0, hi = p.G;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (v.g_first[mid] <= b)
                    lo = mid;
                else
                    hi = mid;
            }
            const int len = min(cap, __ldg(p.lens + b));
            int g = -1;
            if (b >= v.g_first[lo] && b < v.g_first[lo] + v.g_rows[lo] && v.g_len[lo] > 0 &&
                len - (p.L - 1) >= v.g_len[lo]) {
                g = lo;
                atomicMin(&v.g_lead[lo], b);
                atomicAdd(&g_count[lo], 1);
            }
            v.gidx[b] = g;
        }
        __syncthreads();
        // a group of one shares with nobody
        for (int g = threadIdx.x; g < p.G; g += nt)
            if (g_count[g] < 2) v.g_len[g] = 0;
        __syncthreads();
    }
    int64_t units = 0;
    for (int b = threadIdx.x; b < p.B; b += nt) {
        int g = p.G > 0 ? v.gidx[b] : -1;
        if (g >= 0 && v.g_len[g] == 0) g = -1;
        v.gidx[b] = g;
        v.start[b] = g >= 0 ? v.g_len[g] : 0;
        units += own_tiles(p, v, b);
    }
    const int LR = p.L * p.R, own_rt = ceil_div(LR, p.own_rows), KV = p.c.KV;
    units = block_sum(units, tmp) * own_rt * KV;
    // a group's work: tiles of own_kernel, or items of shared_kernel
    auto group_tiles = [&](int g) -> int64_t {
        return p.shared_tc ? 0
                           : (int64_t)ceil_div(v.g_len[g], p.unit_keys) *
                                 ceil_div(v.g_rows[g] * LR, p.own_rows) * KV;
    };
    auto group_items = [&](int g) -> int64_t {
        return p.shared_tc ? (int64_t)ceil_div(v.g_len[g], v.shared_chunk) *
                                 ceil_div(v.g_rows[g] * LR, p.shared_rows)
                           : 0;
    };
    v.shared_chunk = p.shared_unit;
    if (p.G > 0 && p.shared_tc) {
        int64_t n = 0;
        for (int g = threadIdx.x; g < p.G; g += nt)
            n += (int64_t)v.g_len[g] * ceil_div(v.g_rows[g] * LR, p.shared_rows) * KV;
        int64_t want = block_sum(n, tmp) / p.shared_target;
        // one item more than the device holds at once would cost a whole
        // round: chunks grow until all fit (each group has at least one)
        for (int k = 0; k < 8; ++k) {
            want = max((want + p.shared_unit - 1) / p.shared_unit * p.shared_unit,
                       (int64_t)v.shared_chunk + (k > 0 ? p.shared_unit : 0));
            v.shared_chunk = (int)min((int64_t)(1 << 29), want);
            n = 0;
            for (int g = threadIdx.x; g < p.G; g += nt) n += group_items(g) * KV;
            n = block_sum(n, tmp);
            if (n <= p.shared_target || v.shared_chunk >= cap) break;
            want = (int64_t)v.shared_chunk * n / p.shared_target;
        }
    } else if (p.G > 0) {
        int64_t n = 0;
        for (int g = threadIdx.x; g < p.G; g += nt) n += group_tiles(g);
        units += block_sum(n, tmp);
    }
    v.per = max((int64_t)p.own_min, (units + p.own_warps - 1) / p.own_warps);
    // pieces grow until their slots fit the workspace
    auto group_slots = [&](int g) -> int64_t {
        return v.g_rows[g] * (p.shared_tc ? (int64_t)ceil_div(v.g_len[g], v.shared_chunk)
                                          : seg_slots(ceil_div(v.g_len[g], p.unit_keys), v.per));
    };
    for (;;) {
        int64_t n = 0;
        for (int b = threadIdx.x; b < p.B; b += nt) n += seg_slots(own_tiles(p, v, b), v.per);
        for (int g = threadIdx.x; g < p.G; g += nt) n += group_slots(g);
        if (block_sum(n, tmp) <= p.slots || (v.per >= cap && v.shared_chunk >= cap)) break;
        if (v.per < cap) v.per *= 2;
        if (v.shared_chunk < cap) v.shared_chunk *= 2;
    }
    // groups first, then the rows: tiles, slots and items before each
    int64_t tiles_at = 0, slots_at = 0, items_at = 0, all;
    for (int g0 = 0; g0 < p.G; g0 += nt) {
        const int g = g0 + threadIdx.x;
        const bool in = g < p.G;
        const int64_t t = block_scan(in ? group_tiles(g) : 0, &all, tmp);
        if (in) v.g_ubase[g] = tiles_at + t;
        tiles_at += all;
        const int64_t sl = block_scan(in ? group_slots(g) : 0, &all, tmp);
        if (in) v.g_slot[g] = (int)(slots_at + sl);
        slots_at += all;
        const int64_t it = block_scan(in ? group_items(g) : 0, &all, tmp);
        if (in) v.g_items[g] = (int)(items_at + it);
        items_at += all;
    }
    if (threadIdx.x == 0) {
        v.g_ubase[p.G] = tiles_at;
        v.g_items[p.G] = (int)items_at;
    }
    v.shared_items = (int)items_at;
    for (int b0 = 0; b0 < p.B; b0 += nt) {
        const int b = b0 + threadIdx.x;
        const int64_t n = b < p.B ? own_tiles(p, v, b) : 0;
        const int64_t t = block_scan(n * own_rt * KV, &all, tmp);
        if (b < p.B) v.ubase[b] = tiles_at + t;
        tiles_at += all;
        const int64_t sl = block_scan(seg_slots(n, v.per), &all, tmp);
        if (b < p.B) v.sbase[b] = (int)(slots_at + sl);
        slots_at += all;
    }
    if (threadIdx.x == 0) v.ubase[p.B] = tiles_at;
    __syncthreads();
    return v;
}

// For the kernel that adds the slots: `per`, then of each row its own keys'
// first slot, tiles and tiles before, and its group's: first slot, step from
// one piece to the next, chunks (shared_kernel) or tiles, tiles before, row
// tiles a KV head (0: chunks), and the row's place in the group.
constexpr int kDesc = 12;
__host__ __device__ inline size_t desc_bytes(int64_t B) { return 4 * (2 + kDesc * (size_t)B); }

__device__ inline void write_desc(const BatchParams &p, const PlanView &v) {
    if (threadIdx.x == 0) *reinterpret_cast<int64_t *>(p.desc) = v.per;
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
        const int g = v.gidx[b];
        int32_t *d = p.desc + 2 + kDesc * b;
        d[0] = v.sbase[b];
        d[1] = own_tiles(p, v, b);
        *reinterpret_cast<int64_t *>(d + 2) = v.ubase[b];
        d[4] = g >= 0 ? v.g_slot[g] + (b - v.g_first[g]) : 0;
        d[5] = g >= 0 ? v.g_rows[g] : 0;
        *reinterpret_cast<int64_t *>(d + 6) = g >= 0 ? v.g_ubase[g] : 0;
        d[8] = g < 0 ? 0 : p.shared_tc ? ceil_div(v.g_len[g], v.shared_chunk)
                                       : ceil_div(v.g_len[g], p.unit_keys);
        d[9] = g >= 0 && !p.shared_tc ? ceil_div(v.g_rows[g] * p.L * p.R, p.own_rows) : 0;
        d[10] = g >= 0 ? b - v.g_first[g] : 0;
    }
}

// The last index i in [0, n) with base[i] <= x (base ascends, base[0] <= x).
__device__ __forceinline__ int last_at_most(const int64_t *base, int n, int64_t x) {
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

// A piece of work: keys [k0, k1) of table row `row`, for the rows
// [r0, r0 + rows) of sequences from b0 on (row r: sequence b0 + r / (L * R),
// token r / R % L, query head r % R of KV head kv), partial results to slot
// slot0 + r / (L * R).
struct Piece {
    int row, k0, k1, b0, r0, rows, kv, slot0;
};

// shared_kernel's i-th item, i < shared_items * KV: row tiles fastest, so
// that the tiles that read the same keys run together.
__device__ __forceinline__ Piece shared_piece(const BatchParams &p, const PlanView &v, int i) {
    Piece w;
    // item = ((chunk * KV) + kv) * tiles + tile within the group; groups
    // without items have their successor's base: lo ends at the last
    const int KV = p.c.KV;
    int lo = 0, hi = p.G;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)v.g_items[mid] * KV <= i)
            lo = mid;
        else
            hi = mid;
    }
    const int g = lo, rows = v.g_rows[g] * p.L * p.R, tiles = ceil_div(rows, p.shared_rows);
    const int rem = i - v.g_items[g] * KV;
    const int tile = rem % tiles, kc = rem / tiles, kv = kc % KV, chunk = kc / KV;
    w.row = v.g_lead[g];
    w.k0 = chunk * v.shared_chunk;
    w.k1 = min(v.g_len[g], w.k0 + v.shared_chunk);
    w.b0 = v.g_first[g];
    w.r0 = tile * p.shared_rows;
    w.rows = min(p.shared_rows, rows - w.r0);
    w.kv = kv;
    w.slot0 = v.g_slot[g] + chunk * v.g_rows[g];
    return w;
}

// own_kernel: the piece at tile u of the run that ends before tile `end`, run
// `me`, and the tile after the piece.
__device__ __forceinline__ Piece own_piece(const BatchParams &p, const PlanView &v, int64_t u,
                                           int64_t end, int64_t me, bool *is_shared,
                                           int64_t *next) {
    Piece w;
    int rows, tiles, first = 0, step = 1;
    int64_t base;
    *is_shared = u < v.g_ubase[p.G];
    if (*is_shared) {
        const int g = last_at_most(v.g_ubase, p.G, u);
        rows = v.g_rows[g] * p.L * p.R;
        base = v.g_ubase[g];
        step = v.g_rows[g];
        w.row = v.g_lead[g];
        w.b0 = v.g_first[g];
        w.k0 = 0;
        w.k1 = v.g_len[g];
        w.slot0 = v.g_slot[g];
    } else {
        const int b = last_at_most(v.ubase, p.B, u);
        rows = p.L * p.R;
        base = v.ubase[b];
        w.row = w.b0 = b;
        w.k0 = v.start[b];
        w.k1 = min((int)p.key_cap, __ldg(p.lens + b));
        first = w.k0 / p.unit_keys;
        w.slot0 = v.sbase[b];
    }
    tiles = ceil_div(w.k1, p.unit_keys) - first;
    const int rt = ceil_div(rows, p.own_rows);
    const int64_t rem = u - base;
    const int seg = (int)(rem / tiles), at = (int)(rem - (int64_t)seg * tiles);
    const int n = (int)min((int64_t)(tiles - at), end - u);
    w.kv = seg / rt;
    w.r0 = (seg - w.kv * rt) * p.own_rows;
    w.rows = min(p.own_rows, rows - w.r0);
    // a slot (a sequence) for each run that touches the segment
    w.slot0 += (int)(me - (base + (int64_t)seg * tiles) / v.per) * step;
    w.k0 = max(w.k0, (first + at) * p.unit_keys);
    w.k1 = min(w.k1, (first + at + n) * p.unit_keys);
    *next = u + n;
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
