// Attention of a batch over the paged quantised cache: parameters, and the
// plan that its kernels share.
//
// The work of a call is cut into pieces of keys: the shared keys of a group
// (read once for all the group's rows) and each sequence's own keys.  A piece
// leaves, for every row (token, head) it serves, a partial result in a slot of
// the workspace: the largest score (in log2 units), the sum of weights and
// the unnormalised output, fp32.  The slots of a row are added in a fixed
// order afterwards.  All lengths are known to the device only, so a kernel of
// one CTA (plan_kernel) works the pieces out and the others read its tables.
// (Each CTA working them out for itself took 5 to 13 us a kernel.)
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

// The plan's tables, in the workspace.
struct PlanHead {
    int per;           // tiles a warp of own_kernel takes
    int tiles;         // all of them: the groups' (if own_kernel takes those), then the rows'
    int group_tiles;   // the groups'
    int shared_items;  // (chunk, row tile) pairs of shared_kernel, for each KV head
    int shared_chunk;  // keys a chunk
    int pad[3];
};
struct PlanRow {
    int at;            // tiles of own_kernel before this row's own keys
    int tiles;         // of the own keys, for one KV head and row tile
    int k0, k1;        // the own keys
    int slot;          // their first slot
    int group;         // the group that the row shares with, or -1
    int pad[2];
};
struct PlanGroup {
    int at;            // tiles of own_kernel, or items of shared_kernel, before the group
    int pieces;        // of one KV head and row tile: tiles, or chunks
    int len;           // shared keys (0: nobody shares)
    int lead;          // row whose table entries serve them
    int slot;          // first slot
    int first, rows;   // the group's rows
    int pad;
};

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
    PlanHead *head;
    PlanRow *rows;           // [B]
    PlanGroup *groups;       // [G]
    int *runs;               // [own_warps] group (as -1 - g) or row of a run's first tile
    int64_t slots;           // slots of the workspace
    int64_t key_cap;         // max_pages * page, at most 2^24
    int own_rows;            // query rows a tile of own_kernel
    int own_warps;           // its warps
    int own_min;             // tiles a warp takes at least
    int unit_keys;           // keys a tile
    int shared_tc;           // shared_kernel takes the shared keys (else own_kernel)
    int shared_target;       // its CTAs
    int shared_rows;         // query rows a tile of it
    int shared_unit;         // its chunks are multiples of this
    uint32_t *err;
    int withhold;            // test builds only: shared_kernel's first k tile is not announced
};

// A row or group of the plan, past L1.
template <class T>
__device__ __forceinline__ T plan_load(const T *p) {
    static_assert(sizeof(T) == 32, "two 16-byte loads");
    union {
        T t;
        int4 v[2];
    } u;
    u.v[0] = __ldcg(reinterpret_cast<const int4 *>(p));
    u.v[1] = __ldcg(reinterpret_cast<const int4 *>(p) + 1);
    return u.t;
}

__host__ __device__ __forceinline__ int ceil_div(int a, int b) {
    return (int)(((unsigned)a + (unsigned)b - 1u) / (unsigned)b);
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
__device__ __forceinline__ Piece shared_piece(const BatchParams &p, int i) {
    Piece w;
    // item = ((chunk * KV) + kv) * tiles + tile within the group; groups
    // without items have their successor's base: lo ends at the last
    const int KV = p.c.KV;
    int lo = 0, hi = p.G;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.groups[mid].at * KV <= i)
            lo = mid;
        else
            hi = mid;
    }
    const PlanGroup g = p.groups[lo];
    const int chunk_keys = p.head->shared_chunk;
    const int rows = g.rows * p.L * p.R, tiles = ceil_div(rows, p.shared_rows);
    const int rem = i - g.at * KV;
    const int tile = rem % tiles, kc = rem / tiles, kv = kc % KV, chunk = kc / KV;
    w.row = g.lead;
    w.k0 = chunk * chunk_keys;
    w.k1 = min(g.len, w.k0 + chunk_keys);
    w.b0 = g.first;
    w.r0 = tile * p.shared_rows;
    w.rows = min(p.shared_rows, rows - w.r0);
    w.kv = kv;
    w.slot0 = g.slot + chunk * g.rows;
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
