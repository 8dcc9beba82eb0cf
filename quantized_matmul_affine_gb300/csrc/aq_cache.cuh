// Geometry of the paged quantised KV cache, shared by its translation units.
#pragma once

#include "aq_internal.h"

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

}  // namespace aq
