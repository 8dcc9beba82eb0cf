// Geometry of the paged quantised KV cache, shared by its translation units.
#pragma once

#include "aq_paged.h"

#include <atomic>

namespace aq {

// One page holds, for each KV head, a record of `rec` bytes: K codes, V
// codes (side_codes bytes each, rb a row), K and V (scale, bias) pairs
// (side_sb bytes each, `groups` pairs a row).
struct CacheGeom {
    int64_t n_pages;
    int64_t rec;         // bytes of one (page, KV head)
    int64_t page_bytes;  // KV * rec: one page of one layer
    int KV, D, page, page_log2, bits, group;
    int groups;          // D / group
    int rb;              // bytes of one row's codes
    int side_codes;      // page * rb
    int side_sb;         // page * groups * 4
};

inline CacheGeom cache_geom(const aq_cache *c) {
    CacheGeom g;
    g.n_pages = c->n_pages;
    g.KV = (int)c->KV;
    g.D = (int)c->D;
    g.page = c->page;
    g.page_log2 = 0;
    while ((1 << g.page_log2) < c->page) ++g.page_log2;
    g.bits = c->bits;
    g.group = c->group_size;
    g.groups = g.D / g.group;
    g.rb = g.D * g.bits / 8;
    g.side_codes = g.page * g.rb;
    g.side_sb = g.page * g.groups * 4;
    g.rec = 2 * ((int64_t)g.side_codes + g.side_sb);
    g.page_bytes = g.KV * g.rec;
    return g;
}

// The address of a device variable on the current device, looked up once a
// device (a translation unit's one error word: the lookup takes longer than
// a launch).
static inline cudaError_t device_symbol(const uint32_t &symbol, uint32_t **address) {
    static std::atomic<uint32_t *> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    uint32_t *a = known[dev].load(std::memory_order_relaxed);
    if (!a) {
        void *v = nullptr;
        e = cudaGetSymbolAddress(&v, symbol);
        if (e != cudaSuccess) return e;
        a = static_cast<uint32_t *>(v);
        known[dev].store(a, std::memory_order_relaxed);
    }
    *address = a;
    return cudaSuccess;
}

}  // namespace aq
