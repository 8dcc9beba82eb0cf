// Attention of a batch over the paged quantised cache: the kernel that adds
// the pieces' partial results, the choice of kernels and the workspace.
#include "aq_batch_host.cuh"
#include "aq_batch_shared.cuh"

namespace aq {

__device__ uint32_t g_batch_error;

namespace {

// More tiles than a call could have: lens that say so are not real.
constexpr uint64_t kMostTiles = 1u << 30;

constexpr int kPlanThreads = 256;

// The tables of aq_batch.cuh, by one CTA.  What it costs is latency - of its
// loads, barriers and, cold as it is in every call, its own instructions - so
// sums are a warp reduction and a shared-memory add, and what concerns groups
// every warp works out for itself.  10 us by itself with cold caches; a whole
// call over one sequence of 37 tokens takes 9.7 when replayed.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ BatchParams p) {
    extern __shared__ PlanGroup s_g[];                       // [G]
    int *s_n = reinterpret_cast<int *>(s_g + p.G);           // [G] rows that share
    int *s_grp = s_n + p.G;                                  // [B] the row's group, or -1
    int *s_at = s_grp + p.B;                                 // [B] its tiles, then those before it
    __shared__ unsigned s_total, s_warp[2][kPlanThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cap = (int)p.key_cap, LR = p.L * p.R, KV = p.c.KV;
    if (threadIdx.x == 0) s_total = 0;
    launch_dependents();
    grid_dependency_wait();

    // Groups: rows that are long enough for all their tokens to see all
    // shared keys share them; the first of them lends its table entries.
    int disorder = 0;
#pragma unroll 1
    for (int g = threadIdx.x; g < p.G; g += kPlanThreads) {
        const int b0 = p.gstart[g], b1 = p.gstart[g + 1];
        disorder |= b0 < 0 || b1 < b0 || b1 > p.B;
        s_g[g].first = b0;
        s_g[g].rows = b1 - b0;
        s_g[g].len = min(cap, max(0, p.shared[g]));
        s_g[g].lead = p.B;
        s_n[g] = 0;
    }
    disorder = __syncthreads_or(disorder);
    if (disorder) {  // groups that do not ascend within the batch share nothing
        for (int g = threadIdx.x; g < p.G; g += kPlanThreads)
            s_g[g].first = s_g[g].rows = s_g[g].len = 0;
        if (threadIdx.x == 0) atomicOr(p.err, ERR_BATCH_TABLE);
        __syncthreads();
    }
#pragma unroll 1
    for (int b = threadIdx.x; b < p.B; b += kPlanThreads) {
        const int len = min(cap, max(0, p.lens[b]));  // (so that len - L cannot wrap)
        int lo = 0, hi = p.G;
#pragma unroll 1
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_g[mid].first <= b)
                lo = mid;
            else
                hi = mid;
        }
        int g = -1;
        if (p.G > 0 && b >= s_g[lo].first && b < s_g[lo].first + s_g[lo].rows && s_g[lo].len > 0 &&
            len - (p.L - 1) >= s_g[lo].len) {
            g = lo;
            atomicMin(&s_g[g].lead, b);
            atomicAdd(&s_n[g], 1);
        }
        s_grp[b] = g;
        s_at[b] = len;
    }
    __syncthreads();
    // rows: their own keys, and tiles of them
    auto row_of = [&](int b, int len) {
        PlanRow r;
        r.group = s_grp[b];
        if (r.group >= 0 && s_n[r.group] < 2) r.group = -1;  // a group of one shares with nobody
        r.k0 = r.group >= 0 ? s_g[r.group].len : 0;
        r.k1 = max(len, r.k0);
        r.tiles = r.k1 > r.k0 ? ceil_div(r.k1, p.unit_keys) - r.k0 / p.unit_keys : 0;
        return r;
    };
    unsigned n = 0;
#pragma unroll 1
    for (int b = threadIdx.x; b < p.B; b += kPlanThreads) n += row_of(b, s_at[b]).tiles;
    n = __reduce_add_sync(~0u, n);
    if (lane == 0) atomicAdd(&s_total, n);
    __syncthreads();
    const int own_rt = ceil_div(LR, p.own_rows);
    uint64_t units = (uint64_t)s_total * (unsigned)(own_rt * KV);

    // groups: (len x row tiles) summed over them, in units of `each` keys
    const int row_tile = p.shared_tc ? p.shared_rows : p.own_rows;
    auto group_len = [&](int g) { return s_n[g] < 2 ? 0 : s_g[g].len; };
    auto group_units = [&](int each) {
        float sum = 0.f;  // (24 bits are plenty for a choice of size)
#pragma unroll 1
        for (int g = lane; g < p.G; g += 32)
            sum += (float)ceil_div(group_len(g), each) * (float)(ceil_div(s_g[g].rows * LR, row_tile) * KV);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        return sum;
    };
    int chunk = p.shared_unit;
    if (p.G > 0 && p.shared_tc) {
        // Chunks such that all items run at once: one more than the device
        // holds would cost a whole round (each group has at least one).
        float want = group_units(1) / (float)p.shared_target;
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
            chunk = max(chunk + (k ? p.shared_unit : 0),
                        ceil_div((int)fminf(want, 1e9f), p.shared_unit) * p.shared_unit);
            const float items = group_units(chunk);
            if (items <= (float)p.shared_target || chunk >= cap) break;
            want = (float)chunk * items / (float)p.shared_target;
        }
    }
    bool real = units <= kMostTiles;
    if (p.G > 0 && !p.shared_tc) {
        real = real && group_units(p.unit_keys) <= (float)kMostTiles;
        unsigned t = 0;
#pragma unroll 1
        for (int g = lane; g < p.G; g += 32)
            t += ceil_div(group_len(g), p.unit_keys) * ceil_div(s_g[g].rows * LR, row_tile) * KV;
        units += __reduce_add_sync(~0u, t);
    }
    const int per = max(p.own_min, real ? ceil_div((int)units, p.own_warps) : 1);
    // slots that a segment of so many tiles may need: the runs it can touch
    auto seg_slots = [&](int tiles) {
        return tiles > 0 ? (unsigned)(tiles - 1) / (unsigned)per + 2u : 0u;
    };
    // groups first: tiles (or items) and slots before each, by every warp
    unsigned tiles_at = 0, slots_at = 0;
#pragma unroll 1
    for (int g0 = 0; g0 < p.G; g0 += 32) {
        const int g = g0 + lane;
        PlanGroup x = {};
        unsigned t = 0, sl = 0;
        if (g < p.G) {
            x = s_g[g];
            x.len = group_len(g);
            x.pieces = ceil_div(x.len, p.shared_tc ? chunk : p.unit_keys);
            t = x.pieces * ceil_div(x.rows * LR, row_tile) * (p.shared_tc ? 1 : KV);
            sl = x.rows * (p.shared_tc ? x.pieces : seg_slots(x.pieces));
        }
        unsigned bt = t, bs = sl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned u = __shfl_up_sync(~0u, bt, o), w = __shfl_up_sync(~0u, bs, o);
            if (lane >= o) bt += u, bs += w;
        }
        x.at = (int)(tiles_at + bt - t);
        x.slot = (int)(slots_at + bs - sl);
        if (warp == 0 && g < p.G) p.groups[g] = x;
        tiles_at += __shfl_sync(~0u, bt, 31);
        slots_at += __shfl_sync(~0u, bs, 31);
    }
    const int items = p.shared_tc ? (int)tiles_at : 0, group_tiles = p.shared_tc ? 0 : (int)tiles_at;
    tiles_at = group_tiles;
    // then the rows
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        PlanRow r = {};
        unsigned t = 0, sl = 0;
        if (b < p.B) {
            r = row_of(b, s_at[b]);
            if (!real) r.tiles = 0;
            t = r.tiles * own_rt * KV;
            sl = seg_slots(r.tiles);
        }
        unsigned bt = t, bs = sl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned u = __shfl_up_sync(~0u, bt, o), w = __shfl_up_sync(~0u, bs, o);
            if (lane >= o) bt += u, bs += w;
        }
        if (lane == 31) {
            s_warp[0][warp] = bt;
            s_warp[1][warp] = bs;
        }
        __syncthreads();
        unsigned at = tiles_at + bt - t, slot = slots_at + bs - sl;
#pragma unroll 1
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            const unsigned x = s_warp[0][w], y = s_warp[1][w];
            if (w < warp) at += x, slot += y;
            tiles_at += x;
            slots_at += y;
        }
        if (b < p.B) {
            r.at = (int)at;
            r.slot = (int)slot;
            p.rows[b] = r;
            s_at[b] = r.at;
        }
        __syncthreads();
    }
    // the workspace's formula covers every plan; a plan past it does nothing
    real = real && slots_at <= (uint64_t)p.slots;
    if (!real && threadIdx.x == 0) atomicOr(p.err, ERR_BATCH_TABLE);
    if (!real)
        for (int b = threadIdx.x; b < p.B; b += kPlanThreads) {
            p.rows[b].tiles = 0;
            p.rows[b].group = -1;
        }
    const int tiles = real ? (int)tiles_at : 0;
    if (threadIdx.x == 0) {
        PlanHead h = {};
        h.per = per;
        h.tiles = tiles;
        h.group_tiles = group_tiles;
        h.shared_items = real ? items : 0;
        h.shared_chunk = chunk;
        *p.head = h;
    }
    // where each run starts: a warp a group or row writes the runs that start in it
    auto starts = [&](int at, int count, int name) {
#pragma unroll 1
        for (int w = ceil_div(at, per) + lane; (int64_t)w * per < at + count; w += 32) p.runs[w] = name;
    };
    if (!real) return;
    if (!p.shared_tc)
#pragma unroll 1
        for (int g = warp; g < p.G; g += kPlanThreads / 32) {
            const int to = g + 1 < p.G ? p.groups[g + 1].at : group_tiles;
            starts(p.groups[g].at, to - p.groups[g].at, -1 - g);
        }
#pragma unroll 1
    for (int b = warp; b < p.B; b += kPlanThreads / 32)
        starts(s_at[b], (b + 1 < p.B ? s_at[b + 1] : tiles) - s_at[b], b);
}

// A row's output (sequence, token, head): its slots in plan order - the
// shared pieces, then its own - weighted by 2^(max - largest max), 4 (D + 2)
// bytes each.  WPR warps a row: one where there are rows for every warp of the
// device; eight, which take every eighth slot and add up in warp order, where
// a few rows have hundreds of slots each (one row of a 32k-token sequence:
// 200).  A row without slots, or whose keys were all past its limit, is zeros.
// Bound by the latency of its dependent loads: 5120 rows of 128, 24 MB of
// partial results, take 15 us with cold caches, DRAM at 20 %.
template <int D, int WPR>
__global__ void __launch_bounds__(WPR == 1 ? 128 : 32 * WPR)
    join_kernel(const __grid_constant__ BatchParams p) {
    constexpr int kRows = WPR == 1 ? 4 : 1;        // rows a CTA
    constexpr int V = D / 128 > 0 ? D / 128 : 1;   // float4 a lane (half the lanes at D = 64)
    constexpr int kPart = WPR > 1 ? WPR : 1;
    __shared__ float4 part[kPart][D / 4];
    __shared__ float psum[kPart];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = WPR == 1 ? 0 : warp;
    const int64_t row = WPR == 1 ? (int64_t)blockIdx.x * kRows + warp : (int64_t)blockIdx.x;
    const int64_t LH = (int64_t)p.L * p.H;
    if (row >= p.B * LH) {  // whole warps, and only with one warp a row
        grid_dependency_wait();
        return;
    }
    const int b = (int)(row / LH);
    const int lh = (int)(row - b * LH), l = lh / p.H, h = lh - l * p.H;
    const int kv = h / p.R, lr = l * p.R + (h - kv * p.R), LR = p.L * p.R;
    // the plan was complete before the kernel before this one let it start
    const int per = __ldcg(reinterpret_cast<const int *>(p.head));
    const PlanRow d = plan_load(p.rows + b);
    // pieces of a segment of `tiles` tiles from tile u0 on
    auto pieces = [&](int u0, int tiles) {
        return tiles > 0 ? (u0 + tiles - 1) / per - u0 / per + 1 : 0;
    };
    const int own0 = d.slot;
    const int own_n =
        pieces(d.at + (kv * ceil_div(LR, p.own_rows) + lr / p.own_rows) * d.tiles, d.tiles);
    int sh_n = 0, sh0 = 0, sh_step = 0;
    if (d.group >= 0) {
        const PlanGroup g = plan_load(p.groups + d.group);
        const int place = b - g.first;
        sh0 = g.slot + place;
        sh_step = g.rows;
        sh_n = p.shared_tc
                   ? g.pieces
                   : pieces(g.at + (kv * ceil_div(g.rows * LR, p.own_rows) +
                                    (place * LR + lr) / p.own_rows) * g.pieces,
                            g.pieces);
    }
    const int n = sh_n + own_n;
    launch_dependents();
    grid_dependency_wait();
    auto slot_row = [&](int i) -> int64_t {
        const int64_t s = i < sh_n ? sh0 + (int64_t)i * sh_step : own0 + (i - sh_n);
        return s * LH + lh;
    };
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, p.part_ml[slot_row(i)].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
    const float ref = M == -INFINITY ? 0.f : M;
    float4 acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    const bool on = D >= 128 || lane < D / 4;
#pragma unroll 4
    for (int i = sub; i < n; i += WPR) {
        const int64_t at = slot_row(i);
        const float2 ml = p.part_ml[at];
        const float g = batch_ex2(ml.x - ref);
        L = fmaf(ml.y, g, L);
        const float4 *o = reinterpret_cast<const float4 *>(p.part_o + at * D);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float4 v = on ? o[lane + 32 * k] : make_float4(0.f, 0.f, 0.f, 0.f);
            acc[k].x = fmaf(v.x, g, acc[k].x);
            acc[k].y = fmaf(v.y, g, acc[k].y);
            acc[k].z = fmaf(v.z, g, acc[k].z);
            acc[k].w = fmaf(v.w, g, acc[k].w);
        }
    }
    if constexpr (WPR > 1) {
        if (on)
#pragma unroll
            for (int k = 0; k < V; ++k) part[warp][lane + 32 * k] = acc[k];
        if (lane == 0) psum[warp] = L;
        __syncthreads();
        if (warp > 0) return;
        for (int w = 1; w < WPR; ++w) {
            L += psum[w];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if (!on) break;
                const float4 v = part[w][lane + 32 * k];
                acc[k].x += v.x;
                acc[k].y += v.y;
                acc[k].z += v.z;
                acc[k].w += v.w;
            }
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

cudaError_t plan_run(const BatchParams &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, 1, 1);
    cfg.blockDim = dim3(kPlanThreads, 1, 1);
    cfg.dynamicSmemBytes = 8 * (size_t)p.B + (sizeof(PlanGroup) + 4) * (size_t)p.G;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, plan_kernel, p);
}

template <int D>
cudaError_t join_run(const BatchParams &p, cudaStream_t stream) {
    const int64_t rows = (int64_t)p.B * p.L * p.H;
    // eight warps a row while all rows then run at once (16 sequences of 4k
    // tokens, 640 rows: 24.5 us, 29.2 with one; 64 sequences over 8k shared
    // tokens, 2560 rows: 63.8 and 60.4)
    const bool wide = rows <= 8 * (int64_t)num_sms();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(wide ? rows : (rows + 3) / 4), 1, 1);
    cfg.blockDim = dim3(wide ? 256 : 128, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return wide ? cudaLaunchKernelEx(&cfg, join_kernel<D, 8>, p)
                : cudaLaunchKernelEx(&cfg, join_kernel<D, 1>, p);
}

struct BatchPlan {
    int nb, own_rows;      // own_kernel: blocks of 8 query rows, rows a tile
    int own_ctas, unit_keys;
    int row_tiles;         // shared_kernel: tiles of 128 rows a CTA (0: not taken)
    int shared_rows, shared_target;
    // the workspace: the slots' (max, sum), the slots' outputs, the rows' slots
    int64_t slots;
    size_t off_o, off_plan, bytes;
};

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

cudaError_t own_dispatch(const aq_cache *c, const BatchRun &r) {
    if (c->bits == 4)
        return c->D <= 128 ? batch_own4a(c->D, c->group_size, r) : batch_own4b(c->D, c->group_size, r);
    return c->D <= 128 ? batch_own8a(c->D, c->group_size, r) : batch_own8b(c->D, c->group_size, r);
}

BatchPlan plan_for(const aq_cache *c, int64_t B, int64_t L, int64_t H, int64_t G) {
    BatchPlan pl = {};
    const int64_t R = H / c->KV;
    // Rows a KV head that read a group's shared keys, if the groups are even.
    // Up to 16 are one tile of own_kernel, which the tensor core's 128 only beats
    // where there is a group or two (10 rows, 5 heads of 128 at 4 bits over 4k
    // shared tokens: one group 23 us with own_kernel, 18 with shared_kernel;
    // eight groups 44 and 58).  Above it reads the codes once more a tile (25
    // rows in each of eight groups: 78 and 67 us; 20 in each of sixteen at 8
    // bits: 136 and 105).  Two row tiles share the keys' dequantising (160 rows
    // over 8k tokens: 48 us with one, 46 with two).
    const int64_t rows = G > 0 ? B * L * R / G : 0;
    if (c->D <= 256 && rows > 16) pl.row_tiles = c->D <= 128 && rows > 128 ? 2 : 1;
    pl.nb = c->D < 512 && (L * R > 8 || (G > 0 && !pl.row_tiles)) ? 2 : 1;
    pl.own_rows = 8 * pl.nb;
    BatchRun r = {};
    r.nb = pl.nb;
    r.resident = &pl.own_ctas;
    r.unit_keys = &pl.unit_keys;
    if (own_dispatch(c, r) != cudaSuccess || pl.own_ctas < 1) {  // no device: sizes only
        cudaGetLastError();
        pl.own_ctas = 2 * num_sms();
        pl.unit_keys = 16;
    }
    pl.shared_rows = 128 * std::max(1, pl.row_tiles);
    pl.shared_target = num_sms();
    // Slots.  With T runs of own_kernel, a segment of t tiles needs 2 + t / per
    // of them; the segments of all heads and row tiles together make t / per
    // at most T / (heads x row tiles).  A group has a slot a sequence for each
    // piece; shared_kernel makes at most T / (heads x row tiles) + 1.
    const int64_t T = 4 * (int64_t)pl.own_ctas / c->KV + 1;
    const int64_t Ts = (pl.row_tiles ? pl.shared_target : 4 * (int64_t)pl.own_ctas) / c->KV + 2;
    const int64_t per_tile = (pl.row_tiles ? pl.shared_rows : pl.own_rows) / (L * R) + 1;
    pl.slots = 5 * B + T + (G > 0 ? std::min(B, per_tile * G) * Ts : 0);
    const size_t each = (size_t)(pl.slots * L * H);
    pl.off_o = up256(each * sizeof(float2));
    pl.off_plan = pl.off_o + up256(each * (size_t)c->D * sizeof(float));
    pl.bytes = pl.off_plan + sizeof(PlanHead) + (size_t)B * sizeof(PlanRow) +
               (size_t)G * sizeof(PlanGroup) + 16 * (size_t)pl.own_ctas;
    return pl;
}

}  // namespace

bool batch_supported(const aq_cache *c, int64_t L, int64_t H) {
    return L >= 1 && L <= AQ_BATCH_MAX_TOKENS && H % c->KV == 0;
}

size_t batch_workspace_bytes(const aq_cache *c, int64_t B, int64_t L, int64_t H, int64_t G) {
    return plan_for(c, B, L, H, G).bytes;
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
    p.part_o = reinterpret_cast<float *>(ws + pl.off_o);
    p.head = reinterpret_cast<PlanHead *>(ws + pl.off_plan);
    p.rows = reinterpret_cast<PlanRow *>(p.head + 1);
    p.groups = reinterpret_cast<PlanGroup *>(p.rows + a.B);
    p.runs = reinterpret_cast<int *>(p.groups + a.G);
    p.slots = pl.slots;
    p.key_cap = a.max_pages * c->page;
    p.own_rows = pl.own_rows;
    p.unit_keys = pl.unit_keys;
    p.own_min = 64 / pl.unit_keys;
    p.shared_tc = pl.row_tiles > 0;
    p.shared_target = pl.shared_target;
    p.shared_rows = pl.shared_rows;
    p.shared_unit = 128;
    // no more CTAs than the longest sequences there can be give work to
    const int64_t most = p.key_cap / pl.unit_keys + 1, LR = a.L * R;
    const int64_t tiles =
        (a.B * ((LR + pl.own_rows - 1) / pl.own_rows) +
         (a.G > 0 && !pl.row_tiles ? a.B * LR / pl.own_rows + a.G : 0)) * c->KV * most;
    p.own_warps = 4 * (int)std::max<int64_t>(
                          1, std::min<int64_t>(pl.own_ctas, (tiles / p.own_min + 3) / 4));
    cudaError_t e = device_symbol(g_batch_error, &p.err);
    if (e != cudaSuccess) return e;
    e = plan_run(p, a.stream);
    if (e != cudaSuccess) return e;
#ifdef AQ_TEST_HOOKS
    p.withhold = g_test_withhold == 3;
#endif
    if (pl.row_tiles) {
        e = batch_shared(p, pl.row_tiles, num_sms(), a.stream);
        if (e != cudaSuccess) return e;
    }
    r.nb = pl.nb;
    r.stream = a.stream;
    e = own_dispatch(c, r);
    if (e != cudaSuccess) return e;
    switch (c->D) {
        case 64: return join_run<64>(p, a.stream);
        case 128: return join_run<128>(p, a.stream);
        case 256: return join_run<256>(p, a.stream);
        default: return join_run<512>(p, a.stream);
    }
}

cudaError_t batch_read_error(uint32_t *code, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_batch_error, sizeof(uint32_t));
    if (e != cudaSuccess || !clear) return e;
    const uint32_t zero = 0;
    return cudaMemcpyToSymbol(g_batch_error, &zero, sizeof(uint32_t));
}

}  // namespace aq
