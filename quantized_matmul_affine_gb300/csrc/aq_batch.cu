// Attention of a batch over the paged quantised cache: the kernel that adds
// the pieces' partial results, the choice of kernels and the workspace.
#include "aq_batch_host.cuh"
#include "aq_batch_shared.cuh"

namespace aq {

__device__ uint32_t g_batch_error;

namespace {

constexpr int kJoinThreads = 128;

// One warp a row (sequence, token, head): its slots in plan order - the
// shared pieces, then its own - weighted by 2^(max - largest max).  Reads
// 4 (D + 2) bytes a slot; a row without slots, or whose keys were all past
// its limit, is zeros.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ BatchParams p) {
    launch_dependents();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (kJoinThreads / 32) + warp;
    const int64_t LH = (int64_t)p.L * p.H;
    if (row >= p.B * LH) return;
    const int b = (int)(row / LH);
    const int64_t lh = row - b * LH;
    const int32_t *d = p.desc + 5 * b;
    const int own0 = d[0], own_n = d[1], sh0 = d[2], sh_step = d[3], sh_n = d[4];
    const int n = sh_n + own_n;
    auto slot_row = [&](int i) -> int64_t {
        const int64_t s = i < sh_n ? sh0 + (int64_t)i * sh_step : own0 + (i - sh_n);
        return s * LH + lh;
    };
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, p.part_ml[slot_row(i)].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
    const float ref = M == -INFINITY ? 0.f : M;
    constexpr int V = D / 128 > 0 ? D / 128 : 1;  // float4 a lane (half the lanes at D = 64)
    float4 acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    const bool on = D >= 128 || lane < D / 4;
    for (int i = 0; i < n; ++i) {
        const int64_t at = slot_row(i);
        const float2 ml = p.part_ml[at];
        const float g = batch_ex2(ml.x - ref);
        L = fmaf(ml.y, g, L);
        if (!on) continue;
        const float4 *o = reinterpret_cast<const float4 *>(p.part_o + at * D);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float4 v = o[lane + 32 * k];
            acc[k].x = fmaf(v.x, g, acc[k].x);
            acc[k].y = fmaf(v.y, g, acc[k].y);
            acc[k].z = fmaf(v.z, g, acc[k].z);
            acc[k].w = fmaf(v.w, g, acc[k].w);
        }
    }
    if (!on) return;
    // NaN sums stay NaN; only a row that saw nothing is zeros
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        uint2 u;
        const float x = acc[k].x * inv, y = acc[k].y * inv, z = acc[k].z * inv, w = acc[k].w * inv;
        if (p.bf16) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(x, y), c = __floats2bfloat162_rn(z, w);
            u.x = *reinterpret_cast<const uint32_t *>(&a);
            u.y = *reinterpret_cast<const uint32_t *>(&c);
        } else {
            u.x = pack_half2(x, y);
            u.y = pack_half2(z, w);
        }
        reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + row * D)[lane + 32 * k] = u;
    }
}

// Workspace: the slots' (max, sum), the slots' outputs, the rows' slots.
struct BatchWs {
    int64_t slots;
    size_t off_o, off_desc, bytes;
};

struct BatchPlan {
    int nb, own_rows;      // own-keys kernel: blocks of 8 query rows, rows a tile
    int row_tiles;         // shared keys on the tensor core: tiles a CTA (0: not)
    int shared_rows;       // rows a tile of the kernel that takes shared keys
    int own_target, shared_target;
    BatchWs ws;
};

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

cudaError_t own_dispatch(const aq_cache *c, const BatchRun &r);

// CTAs of the own-keys kernel the device holds at once (2 a SM without one).
int resident_ctas(const aq_cache *c, int64_t B, int64_t G, int nb) {
    int n = 0;
    BatchRun r = {};
    r.prm.B = (int)B;
    r.prm.G = (int)G;
    r.nb = nb;
    r.resident = &n;
    if (own_dispatch(c, r) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return 2 * num_sms();
    }
    return n;
}

BatchPlan plan_for(const aq_cache *c, int64_t B, int64_t L, int64_t H, int64_t G) {
    BatchPlan pl = {};
    const int64_t R = H / c->KV;
    // rows a KV head that read a group's shared keys, if the batch is one of
    // even groups
    const int64_t rows = G > 0 ? B * L * R / G : 0;
    if (c->D <= 256 && rows > 32) pl.row_tiles = c->D <= 128 && rows > 128 ? 2 : 1;
    pl.nb = c->D < 512 && (L * R > 8 || (G > 0 && !pl.row_tiles)) ? 2 : 1;
    pl.own_rows = 8 * pl.nb;
    pl.shared_rows = pl.row_tiles ? 128 * pl.row_tiles : pl.own_rows;
    pl.own_target = resident_ctas(c, B, G, pl.nb);
    pl.shared_target = pl.row_tiles ? num_sms() : pl.own_target;
    // Slots.  With T pieces x row tiles x heads wanted, own keys make at most
    // T / heads + B pieces; a group's shared keys make at most T / (heads *
    // its row tiles) + 1 pieces, one slot a sequence of the group each.
    const int64_t T = pl.own_target / c->KV + 1, Ts = pl.shared_target / c->KV + 1;
    const int64_t per_tile = pl.shared_rows / (L * R) + 1;  // sequences a tile
    pl.ws.slots = 3 * B + T + (G > 0 ? std::min(B, per_tile * G) * Ts : 0);
    const size_t each = (size_t)(pl.ws.slots * L * H);
    pl.ws.off_o = up256(each * sizeof(float2));
    pl.ws.off_desc = pl.ws.off_o + up256(each * (size_t)c->D * sizeof(float));
    pl.ws.bytes = pl.ws.off_desc + up256((size_t)B * 5 * sizeof(int32_t));
    return pl;
}

cudaError_t own_dispatch(const aq_cache *c, const BatchRun &r) {
    if (c->bits == 4)
        return c->D <= 128 ? batch_own4a(c->D, c->group_size, r) : batch_own4b(c->D, c->group_size, r);
    return c->D <= 128 ? batch_own8a(c->D, c->group_size, r) : batch_own8b(c->D, c->group_size, r);
}

}  // namespace

bool batch_supported(const aq_cache *c, int64_t L, int64_t H) {
    return L >= 1 && L <= AQ_BATCH_MAX_TOKENS && H % c->KV == 0;
}

size_t batch_workspace_bytes(const aq_cache *c, int64_t B, int64_t L, int64_t H, int64_t G) {
    return plan_for(c, B, L, H, G).ws.bytes;
}

cudaError_t batch_launch(const aq_cache *c, int64_t layer, const BatchArgs &a) {
    const int64_t R = a.H / c->KV;
    const BatchPlan pl = plan_for(c, a.B, a.L, a.H, a.G);
    BatchRun r = {};
    BatchParams &p = r.prm;
    p.c = cache_geom(c);
    p.layer = static_cast<const uint8_t *>(c->pool_dev) + layer * c->n_pages * p.c.page_bytes;
    p.q = a.q;
    p.out = a.out;
    p.q_stride = a.q_stride;
    p.table = a.table;
    p.lens = a.lens;
    p.gstart = a.group_start;
    p.shared = a.shared;
    p.max_pages = a.max_pages;
    p.B = (int)a.B;
    p.L = (int)a.L;
    p.H = (int)a.H;
    p.R = (int)R;
    p.G = (int)a.G;
    p.bf16 = a.dtype == AQ_BF16;
    p.scale2 = a.scale * 1.4426950408889634f;
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    p.part_ml = reinterpret_cast<float2 *>(ws);
    p.part_o = reinterpret_cast<float *>(ws + pl.ws.off_o);
    p.desc = reinterpret_cast<int32_t *>(ws + pl.ws.off_desc);
    p.slots = pl.ws.slots;
    p.key_cap = a.max_pages * c->page;
    p.own_target = pl.own_target;
    p.own_rows = pl.own_rows;
    p.own_unit = 128;
    p.shared_target = pl.shared_target;
    p.shared_rows = pl.shared_rows;
    p.shared_unit = 128;
    void *err = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&err, g_batch_error);
    if (e != cudaSuccess) return e;
    p.err = static_cast<uint32_t *>(err);
    if (pl.row_tiles) {
        e = batch_shared(p, pl.row_tiles, num_sms(), a.stream);
        if (e != cudaSuccess) return e;
    }
    r.do_shared = !pl.row_tiles;
    r.nb = pl.nb;
    r.stream = a.stream;
    const int64_t pieces = (p.key_cap + p.own_unit - 1) / p.own_unit;
    const int64_t tiles = (a.L * R + pl.own_rows - 1) / pl.own_rows;
    r.max_items = (a.B * pieces * tiles +
                   (r.do_shared && a.G > 0 ? (a.B * a.L * R / pl.own_rows + a.G) * pieces : 0)) *
                  c->KV;
    e = own_dispatch(c, r);
    if (e != cudaSuccess) return e;
    const int64_t rows = a.B * a.L * a.H;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32)), 1, 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.stream = a.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    switch (c->D) {
        case 64: return cudaLaunchKernelEx(&cfg, join_kernel<64>, p);
        case 128: return cudaLaunchKernelEx(&cfg, join_kernel<128>, p);
        case 256: return cudaLaunchKernelEx(&cfg, join_kernel<256>, p);
        default: return cudaLaunchKernelEx(&cfg, join_kernel<512>, p);
    }
}

cudaError_t batch_read_error(uint32_t *code, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_batch_error, sizeof(uint32_t));
    if (e != cudaSuccess || !clear) return e;
    const uint32_t zero = 0;
    return cudaMemcpyToSymbol(g_batch_error, &zero, sizeof(uint32_t));
}

}  // namespace aq
