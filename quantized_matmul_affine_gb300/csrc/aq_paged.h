// Host-side declarations of the paged cache and the attention over it.
#pragma once

#include "aq_internal.h"

namespace aq {

// Device-side error codes, as in aq_internal.h.
enum : uint32_t {
    ERR_CACHE_TABLE = 0x0105,  // a page table names a page outside the pool
    ERR_BATCH_BASE = 0x0006,   // waits of the batch attention
    ERR_BATCH_TABLE = 0x0106,  // its page table names a page outside the pool, or its groups or lens
                               // cannot be
};

// The paged cache (aq_cache.cu); arguments checked by the entry points.
struct CacheTables {
    const int32_t *refs_in, *table_in, *lens_in;
    int32_t *refs, *table, *lens;
    const int32_t *arg0, *arg1;
    int32_t *status, *ws;
    int64_t B, max_pages;
};
// k (or v) null: reads rows into k_out, v_out; otherwise appends.
cudaError_t cache_append_launch(const aq_cache *c, int64_t layer, int dtype, const void *k,
                                int64_t k_stride, const void *v, int64_t v_stride, void *k_out,
                                void *v_out, int64_t T, const int32_t *cu, const int32_t *start,
                                const int32_t *table, int64_t B, int64_t max_pages,
                                cudaStream_t stream);
cudaError_t cache_fork_launch(const aq_cache *c, const CacheTables &t, cudaStream_t stream);
cudaError_t cache_trim_launch(const aq_cache *c, const CacheTables &t, cudaStream_t stream);
cudaError_t cache_grow_launch(const aq_cache *c, const CacheTables &t, cudaStream_t stream);
cudaError_t cache_compact_launch(const aq_cache *c, const CacheTables &t, cudaStream_t stream);
cudaError_t cache_copy_launch(const aq_cache *c, const int32_t *src, const int32_t *dst, int64_t n,
                              cudaStream_t stream);
// Attention of a batch over the paged cache (aq_batch.cu).
struct BatchArgs {
    int dtype;
    const void *q;
    int64_t q_stride;  // elements from one token's heads to the next's
    const int32_t *table, *lens, *group_start, *shared;
    int64_t B, L, H, G, max_pages;
    float scale;
    void *out, *ws;
    size_t ws_bytes;
    cudaStream_t stream;
};
bool batch_supported(const aq_cache *c, int64_t L, int64_t H);
size_t batch_workspace_bytes(const aq_cache *c, int64_t B, int64_t L, int64_t H, int64_t G);
cudaError_t batch_launch(const aq_cache *c, int64_t layer, const BatchArgs &a);

cudaError_t cache_read_error(uint32_t *code, bool clear);
cudaError_t batch_read_error(uint32_t *code, bool clear);

}  // namespace aq
