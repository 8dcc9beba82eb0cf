// The paged quantised KV cache: quantising rows into pages, reading rows
// back, and the page tables' operations (fork, grow, trim, compact, copy).
//
// A pool is pages [layers][n_pages][KV][record]; the record of one page and
// one KV head holds P cached rows of K and V in the affine format:
//   K codes [P][D*bits/8 bytes] | V codes [P][D*bits/8 bytes] |
//   K (scale, bias) fp16 pairs [P][D/group] | V (scale, bias) [P][D/group].
// One page and head is one contiguous piece, so the attention reads it as
// one stream and a page moves as one block a layer.
#include "aq_internal.h"
#include "aq_ptx.cuh"
#include "aq_cache.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

namespace aq {

__device__ uint32_t g_cache_error;

namespace {

// ---------------------------------------------------------------------------
// Rows in and out.
// ---------------------------------------------------------------------------

struct RowParams {
    CacheGeom c;
    uint8_t *layer;           // the layer's pages
    const void *in[2];        // append: k, v
    int64_t in_stride[2];     // elements from one token to the next
    void *out[2];             // read: k, v, dense [T][KV][D]
    const int32_t *cu, *start, *table;
    int64_t T;
    int B;
    int span;                 // lanes a token
    int each;                 // tokens they take one after another
    int head_log2, lane_log2;  // lanes a head (D / 8) and a group (group / 8)
    int64_t max_pages;
    uint32_t *err;
};

// The sequence b with cu[b] <= t < cu[b + 1] (cu ascends), or -1.
__device__ __forceinline__ int find_row(const int32_t *cu, int B, int t) {
    int lo = 0, hi = B;  // the answer, if any, is in [lo, hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return cu[lo] <= t && t < cu[lo + 1] ? lo : -1;
}

// The record of token t's page and KV head 0, its slot in the page; nullptr
// where the token has no place (padding, or a table that names none: the
// latter sets the error word).
__device__ __forceinline__ uint8_t *token_record(const RowParams &p, int t, int *slot) {
    const int b = find_row(p.cu, p.B, t);
    if (b < 0) return nullptr;
    const int64_t pos = (int64_t)p.start[b] + (t - p.cu[b]);
    const int64_t pg = pos >> p.c.page_log2;
    if (pos < 0 || pg >= p.max_pages) {
        atomicOr(p.err, ERR_CACHE_TABLE);
        return nullptr;
    }
    const int64_t id = p.table[(int64_t)b * p.max_pages + pg];
    if (id < 0 || id >= p.c.n_pages) {
        atomicOr(p.err, ERR_CACHE_TABLE);
        return nullptr;
    }
    *slot = (int)(pos & (p.c.page - 1));
    return p.layer + id * p.c.page_bytes;
}

template <bool BF16>
__device__ __forceinline__ void widen(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
}

constexpr int kRowThreads = 128;
constexpr int kRowLoads = 4;  // 16-byte loads a lane has under way

// One lane takes 8 values (a 16-byte load), `p.span` lanes (8, 16 or 32: the
// most that divide a token's lanes) take a token and look up its page once;
// the GROUP / 8 lanes of a group reduce min and max by shuffles.  The
// quantiser's rule is aq_quantize_ex's (codes of the IEEE quotient, by the
// reciprocal-and-check form of aq_quant.cu).  blockIdx.y: K or V.
//
// Bytes: 2 a value in, bits / 8 and a pair a group out - 12.7 us at 16k bf16
// tokens of 8 heads of 128 to 4 bits, where it takes 36.  The issue slots are
// 73 % taken (a value costs a clamp, two fused steps and a shifted add, a
// group six shuffles), DRAM 25 %: bound by instructions, and in a decode step
// (64 tokens) by its chain of loads, 3 to 4 us.
template <int BITS, bool BF16>
__global__ void __launch_bounds__(kRowThreads) append_kernel(const __grid_constant__ RowParams p) {
    constexpr int kQmax = (1 << BITS) - 1;
    const int which = blockIdx.y;
    const int per_token = p.c.KV * p.c.D / 8, lanes = p.c.group / 8;
    const int at = (int)(threadIdx.x % p.span);
    const int t0 = (int)(blockIdx.x * (kRowThreads / p.span) + threadIdx.x / p.span) * p.each;
    // lane i looks up the page of the i-th of these tokens, for all of them
    int my_slot = 0;
    uint8_t *my_rec = nullptr;
    if (at < p.each && t0 + at < p.T) my_rec = token_record(p, t0 + at, &my_slot);
    const int lead = (int)(threadIdx.x & 31) - at;
#pragma unroll 1
    for (int i = 0; i < p.each; ++i) {
        const int t = t0 + i;
        const int slot = __shfl_sync(~0u, my_slot, lead + i);
        uint8_t *rec = reinterpret_cast<uint8_t *>(
            __shfl_sync(~0u, reinterpret_cast<unsigned long long>(my_rec), lead + i));
        const uint4 *in = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.in[which]) +
                                                          (int64_t)t * p.in_stride[which]);
        uint8_t *codes = rec + which * p.c.side_codes + slot * p.c.rb;
        __half2 *pairs = reinterpret_cast<__half2 *>(rec + 2 * p.c.side_codes + which * p.c.side_sb) +
                         slot * p.c.groups;
        for (int e0 = 0; e0 < per_token; e0 += kRowLoads * p.span) {
            uint4 raw[kRowLoads];
#pragma unroll
            for (int k = 0; k < kRowLoads; ++k) {
                const int e = e0 + k * p.span + at;
                raw[k] = rec && e < per_token ? in[e] : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int k = 0; k < kRowLoads; ++k) {
                const int e = e0 + k * p.span + at;
                if (e0 + k * p.span >= per_token) break;  // alike for all lanes
                float f[8];
                widen<BF16>(raw[k], f);
                float lo = f[0], hi = f[0];
#pragma unroll
                for (int j = 1; j < 8; ++j) {
                    lo = fminf(lo, f[j]);
                    hi = fmaxf(hi, f[j]);
                }
#pragma unroll
                for (int o = 1; o < 16; o <<= 1)
                    if (o < lanes) {
                        lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
                        hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
                    }
                const __half s16 = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), (float)kQmax));
                const __half b16 = __float2half_rn(lo);
                const float s = __half2float(s16), b = __half2float(b16);
                // Adding 1.5 * 2^23 rounds to an integer, which is then the low bits
                // of the sum: codes are gathered by shifted adds of the sums' bits,
                // less what the magic number's own bits add up to.
                constexpr float kMagic = 12582912.0f;
                constexpr int kWords = BITS / 4, kCodes = 32 / BITS;
                constexpr uint32_t kOnes = BITS == 4 ? 0x11111111u : 0x01010101u;
                // the product with the rounded reciprocal is within 1.5 * 2^-23
                // relative of the IEEE quotient: this much of an integer and a half
                constexpr float kEdge = BITS == 4 ? 3.0517578125e-05f : 4.8828125e-04f;
                const float r = __frcp_rn(s);
                const float2 r2 = make_float2(r, r), b2 = make_float2(-b, -b);
                const float2 m2 = make_float2(kMagic, kMagic), n2 = make_float2(-kMagic, -kMagic);
                uint32_t w[kWords];
                float far = 0.f;  // from the nearest integer
#pragma unroll
                for (int u = 0; u < kWords; ++u) w[u] = 0u - (kOnes * __float_as_uint(kMagic));
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    float2 q = __fmul2_rn(__fadd2_rn(make_float2(f[j], f[j + 1]), b2), r2);
                    q.x = fminf(fmaxf(q.x, 0.f), (float)kQmax);
                    q.y = fminf(fmaxf(q.y, 0.f), (float)kQmax);
                    const float2 m = __fadd2_rn(q, m2);
                    const float2 d = __ffma2_rn(__fadd2_rn(m, n2), make_float2(-1.f, -1.f), q);
                    far = fmaxf(far, fmaxf(fabsf(d.x), fabsf(d.y)));
                    w[j / kCodes] += __float_as_uint(m.x) << (j % kCodes * BITS);
                    w[j / kCodes] += __float_as_uint(m.y) << ((j + 1) % kCodes * BITS);
                }
                if (far > 0.5f - kEdge) {  // near a tie: by the quotient itself
#pragma unroll
                    for (int u = 0; u < kWords; ++u) w[u] = 0u;
#pragma unroll 1
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t h = reinterpret_cast<const uint32_t *>(&raw[k])[j / 2];
                        const float v = BF16 ? __uint_as_float(j & 1 ? h & 0xFFFF0000u : h << 16)
                                             : __half2float(__ushort_as_half((uint16_t)(h >> (16 * (j & 1)))));
                        const float q =
                            fminf(fmaxf(__fdiv_rn(__fsub_rn(v, b), s), 0.f), (float)kQmax);
                        const uint32_t code = __float_as_uint(__fadd_rn(q, kMagic)) & (uint32_t)kQmax;
                        if (kWords == 1 || j < kCodes)
                            w[0] |= code << (j % kCodes * BITS);
                        else
                            w[kWords - 1] |= code << (j % kCodes * BITS);
                    }
                }
                if (s == 0.f)
#pragma unroll
                    for (int u = 0; u < kWords; ++u) w[u] = 0u;
                if (!rec) continue;
                const int kv = e >> p.head_log2, d8 = e & ((1 << p.head_log2) - 1);
                uint32_t *dst = reinterpret_cast<uint32_t *>(codes + kv * p.c.rec) + d8 * (BITS / 4);
                if constexpr (BITS == 4)
                    *dst = w[0];
                else
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[kWords - 1]);
                if ((d8 & (lanes - 1)) == 0)
                    reinterpret_cast<__half2 *>(reinterpret_cast<uint8_t *>(pairs) +
                                                kv * p.c.rec)[d8 >> p.lane_log2] = __halves2half2(s16, b16);
            }
        }
    }
}

// The reverse, shared out alike: one lane turns 8 codes into 8 values of the
// output type, each scale * code + bias in one fp32 fma (the product is exact)
// and one rounding.  16k tokens as above: 20 us against 12.7 of traffic, the
// issue slots 70 % taken (a shift, a mask, an add and an fma a value).
template <int BITS, bool BF16>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const __grid_constant__ RowParams p) {
    const int which = blockIdx.y;
    const int per_token = p.c.KV * p.c.D / 8;
    const int at = (int)(threadIdx.x % p.span);
    const int t0 = (int)(blockIdx.x * (kRowThreads / p.span) + threadIdx.x / p.span) * p.each;
    int my_slot = 0;
    const uint8_t *my_rec = nullptr;
    if (at < p.each && t0 + at < p.T) my_rec = token_record(p, t0 + at, &my_slot);
    const int lead = (int)(threadIdx.x & 31) - at;
#pragma unroll 1
    for (int i = 0; i < p.each; ++i) {
        const int t = t0 + i;
        const int slot = __shfl_sync(~0u, my_slot, lead + i);
        const uint8_t *rec = reinterpret_cast<const uint8_t *>(
            __shfl_sync(~0u, reinterpret_cast<unsigned long long>(my_rec), lead + i));
        if (t >= p.T) continue;
        const uint8_t *codes = rec + which * p.c.side_codes + slot * p.c.rb;
        const uint8_t *pairs = rec + 2 * p.c.side_codes + which * p.c.side_sb + slot * p.c.groups * 4;
        uint4 *out = static_cast<uint4 *>(p.out[which]) + (int64_t)t * per_token;
        for (int e0 = at; e0 < per_token; e0 += kRowLoads * p.span) {
            uint32_t w[kRowLoads][2];
            __half2 sb[kRowLoads];
#pragma unroll
            for (int k = 0; k < kRowLoads; ++k) {
                const int e = e0 + k * p.span;
                w[k][0] = w[k][1] = 0u;
                sb[k] = __float2half2_rn(0.f);
                if (!rec || e >= per_token) continue;
                const int kv = e >> p.head_log2, d8 = e & ((1 << p.head_log2) - 1);
                const uint32_t *src =
                    reinterpret_cast<const uint32_t *>(codes + kv * p.c.rec) + d8 * (BITS / 4);
                if constexpr (BITS == 4) {
                    w[k][0] = *src;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2 *>(src);
                    w[k][0] = v.x;
                    w[k][1] = v.y;
                }
                sb[k] = reinterpret_cast<const __half2 *>(pairs + kv * p.c.rec)[d8 >> p.lane_log2];
            }
#pragma unroll
            for (int k = 0; k < kRowLoads; ++k) {
                const int e = e0 + k * p.span;
                if (e >= per_token) break;
                const float2 f = __half22float2(sb[k]);
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float v[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int bit = (2 * j + h) * BITS;
                        const uint32_t code = (w[k][bit / 32] >> (bit % 32)) & ((1u << BITS) - 1u);
                        // 2^23 + code, less 2^23: the code as a float
                        v[h] = fmaf(__uint_as_float(0x4B000000u | code) - 8388608.f, f.x, f.y);
                    }
                    if constexpr (BF16) {
                        const __nv_bfloat162 x = __floats2bfloat162_rn(v[0], v[1]);
                        o[j] = *reinterpret_cast<const uint32_t *>(&x);
                    } else {
                        o[j] = pack_half2(v[0], v[1]);
                    }
                }
                out[e] = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Page tables.  Each operation is one launch of one thread-block cluster:
// its CTAs share the rows and the pages, the cluster barrier separates the
// steps, so nothing is done by a page or row count that the host would have
// to know, and a call can be captured and replayed.  All are latency: cluster
// barriers, dependent loads and the launch (512 rows of 2300 tokens in
// pages of 64: fork 6.5, trim 8, grow 11 us; compact over 8192 pages 10.5).
// ---------------------------------------------------------------------------

constexpr int kCtas = 8;        // a portable cluster
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCopyBits = 16;   // of a packed (pages, copies)

struct TableParams {
    const int32_t *refs_in, *table_in, *lens_in;
    int32_t *refs, *table, *lens;
    const int32_t *arg0, *arg1;  // parent and keep, add, or keep
    int32_t *status;
    int32_t *ws;
    int64_t n_pages, max_pages;
    int B, page, page_log2;
};

__device__ __forceinline__ int pages_of(int len, int log2) {
    return (int)(((int64_t)len + (1 << log2) - 1) >> log2);
}

// refs, table and lens into the output arrays where those are others.
__device__ __forceinline__ void carry_over(const TableParams &p, int rank) {
    const int64_t step = (int64_t)kCtas * kThreads, at = (int64_t)rank * kThreads + threadIdx.x;
    if (p.refs != p.refs_in)
        for (int64_t i = at; i < p.n_pages; i += step) p.refs[i] = p.refs_in[i];
    if (p.table != p.table_in)
        for (int64_t i = at; i < (int64_t)p.B * p.max_pages; i += step)
            p.table[i] = p.table_in[i];
    if (p.lens != p.lens_in)
        for (int64_t i = at; i < p.B; i += step) p.lens[i] = p.lens_in[i];
}

// A row's length as the operations take it: never past its table's width.
__device__ __forceinline__ bool sound_len(const TableParams &p, int len) {
    return len >= 0 && pages_of(len, p.page_log2) <= p.max_pages;
}

// Sum over the cluster of one int per CTA: every CTA writes its value to all
// of them (slot[rank]); complete after the next cluster barrier.
__device__ __forceinline__ void publish(int *slot, int rank, int value) {
    const uint32_t a = smem_u32(slot + rank);
    for (int r = 0; r < kCtas; ++r)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_rank(a, (uint32_t)r)),
                     "r"(value)
                     : "memory");
}

// The pages of warp w of this CTA: a contiguous run, a multiple of 32 long.
struct Run {
    int64_t begin, end;
};
__device__ __forceinline__ Run warp_run(const TableParams &p, int rank) {
    const int64_t each = ((p.n_pages + kCtas * kWarps - 1) / (kCtas * kWarps) + 31) / 32 * 32;
    const int64_t w = (int64_t)rank * kWarps + (threadIdx.x >> 5);
    Run r;
    r.begin = min(p.n_pages, w * each);
    r.end = min(p.n_pages, r.begin + each);
    return r;
}

// Pages of the run that are live (refs > 0); the loads of eight steps are in
// flight together.
__device__ __forceinline__ int count_live(const int32_t *refs, Run r) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int64_t i = r.begin + lane; i < r.end; i += 256) {
        int v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = i + 32 * j < r.end ? refs[i + 32 * j] : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) n += v[j] > 0;
    }
    return __reduce_add_sync(~0u, n);
}

// Fork: row b with parent[b] >= 0 (b empty) becomes a copy of that row's
// first keep[b] tokens (all of them for keep[b] < 0): the same pages, counted
// once more.  A bad row (a parent outside the batch, b itself or another
// child, a row that is not empty, more tokens than the parent has) is counted
// in status[1], and then nothing changes.
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads) fork_kernel(
    const TableParams p) {
    __shared__ int s_bad;
    __shared__ unsigned long long s_pages[kWarps];  // together they may pass 32 bits
    const int rank = (int)cluster_ctarank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    launch_dependents();
    grid_dependency_wait();
    carry_over(p, rank);
    if (rank == 0 && threadIdx.x < 4) p.status[threadIdx.x] = 0;
    int bad = 0;
    unsigned long long pages = 0;
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const int par = p.arg0[b], len = p.lens_in[b];
        if (par < 0) continue;
        bool ok = par < p.B && par != b && len == 0 && p.arg0[par] < 0;
        if (ok) {
            const int plen = p.lens_in[par], keep = p.arg1[b] < 0 ? plen : p.arg1[b];
            ok = keep <= plen && sound_len(p, plen);
            if (ok) pages += pages_of(keep, p.page_log2);
        }
        bad += !ok;
    }
    if (bad) atomicAdd(&s_bad, bad);
    for (int o = 16; o >= 1; o >>= 1) pages += __shfl_xor_sync(~0u, pages, o);
    if (lane == 0) s_pages[warp] = pages;
    // every CTA has counted the same rows; what was carried over is in place
    // cluster-wide before a count or an entry changes
    cluster_sync();
    const bool none = s_bad != 0;
    if (!none)
        for (int b = rank * kWarps + warp; b < p.B; b += kCtas * kWarps) {
            const int par = p.arg0[b];
            if (par < 0) continue;
            const int plen = p.lens_in[par], keep = p.arg1[b] < 0 ? plen : p.arg1[b];
            const int n = pages_of(keep, p.page_log2);
            for (int i = lane; i < n; i += 32) {
                const int id = p.table_in[(int64_t)par * p.max_pages + i];
                p.table[(int64_t)b * p.max_pages + i] = id;
                if (id >= 0 && id < p.n_pages)
                    atomicAdd(&p.refs[id], 1);
                else
                    atomicMax(&p.status[0], 3);
            }
            if (lane == 0) p.lens[b] = keep;  // b is no row's parent
        }
    if (rank == 0 && threadIdx.x == 0) {
        if (none) atomicMax(&p.status[0], 2);
        p.status[1] = s_bad;
        unsigned long long all = 0;
        for (int w = 0; w < kWarps; ++w) all += s_pages[w];
        p.status[2] = none ? 0 : (int)min(all, (unsigned long long)INT32_MAX);
    }
}

// Trim: row b with 0 <= keep[b] < lens[b] gives back the pages past its
// first keep[b] tokens (0: all of them).  status[2]: pages that became free.
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads) trim_kernel(
    const TableParams p) {
    const int rank = (int)cluster_ctarank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ int s_bad;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    launch_dependents();
    grid_dependency_wait();
    carry_over(p, rank);
    if (rank == 0 && threadIdx.x < 4) p.status[threadIdx.x] = 0;
    int bad = 0;
    for (int b = threadIdx.x; b < p.B; b += kThreads)
        bad += p.arg0[b] >= 0 && !sound_len(p, p.lens_in[b]);
    if (bad) atomicAdd(&s_bad, bad);
    cluster_sync();
    const bool none = s_bad != 0;
    int freed = 0;
    if (!none)
        for (int b = rank * kWarps + warp; b < p.B; b += kCtas * kWarps) {
            const int keep = p.arg0[b], len = p.lens_in[b];
            if (keep < 0 || keep >= len) continue;
            const int n0 = pages_of(keep, p.page_log2), n1 = pages_of(len, p.page_log2);
            for (int i = n0 + lane; i < n1; i += 32) {
                int32_t *at = p.table + (int64_t)b * p.max_pages + i;
                const int id = *at;
                *at = -1;
                if (id >= 0 && id < p.n_pages)
                    freed += atomicSub(&p.refs[id], 1) == 1;
                else
                    atomicMax(&p.status[0], 3);
            }
            __syncwarp();
            if (lane == 0) p.lens[b] = keep;
        }
    freed = __reduce_add_sync(~0u, freed);
    if (lane == 0 && freed) atomicAdd(&p.status[2], freed);
    if (rank == 0 && threadIdx.x == 0) {
        if (none) atomicMax(&p.status[0], 2);
        p.status[1] = s_bad;
    }
}

// Grow: every row gets pages for add[b] more tokens, the lowest free pages
// in row order.  A row whose last page is partly filled and shared gets a
// page of its own first (the copy is made by copy_rows_kernel), unless all
// the page's holders grow in this call and it is the last of them.  Too few
// free pages (status 1, how many are missing) or bad rows (status 2, how
// many): nothing changes.  status[2] pages taken, status[3] copies.
//
// ws: [0] number of copies, then (source, target, rows) of each, then one
// int a row.
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads) grow_kernel(
    const TableParams p) {
    extern __shared__ int s_rows[];  // [3][B]: shared last page, pages before, copies before
    int *s_page = s_rows, *s_base = s_rows + p.B, *s_copy = s_rows + 2 * p.B;
    __shared__ int s_bad, s_free[kCtas], s_warp[kWarps];
    __shared__ long long s_scan[kWarps];
    const int rank = (int)cluster_ctarank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    // the cluster's CTAs write to each other's s_free: all have started
    cluster_sync();
    launch_dependents();
    grid_dependency_wait();
    carry_over(p, rank);
    if (rank == 0 && threadIdx.x < 4) p.status[threadIdx.x] = 0;
    int32_t *list = p.ws + 1, *flag = p.ws + 1 + 3 * (int64_t)p.B;
    const int mask = p.page - 1;

    const Run run = warp_run(p, rank);
    const int nfree = (int)(run.end - run.begin) - count_live(p.refs_in, run);
    if (lane == 0) s_warp[warp] = nfree;
    int bad = 0, outside = 0;
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const int len = p.lens_in[b], add = p.arg0[b];
        const bool ok = add >= 0 && sound_len(p, len) && add <= INT32_MAX - len &&
                        pages_of(len + add, p.page_log2) <= p.max_pages;
        bad += !ok;
        int page = -1;
        if (ok && add > 0 && (len & mask)) {
            const int id = p.table_in[(int64_t)b * p.max_pages + (len >> p.page_log2)];
            if (id < 0 || id >= p.n_pages)
                outside = 1;
            else if (p.refs_in[id] > 1)
                page = id;
        }
        s_page[b] = page;
    }
    if (bad) atomicAdd(&s_bad, bad);
    __syncthreads();
    if (warp == 0) {
        int n = s_warp[lane], before = n;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(~0u, before, o);
            if (lane >= o) before += v;
        }
        s_warp[lane] = before - n;
        if (lane == 31) publish(s_free, rank, before);
    }
    for (int b = rank * kWarps + warp; b < p.B; b += kCtas * kWarps) {
        const int page = s_page[b];
        int copy = 0;
        if (page >= 0) {
            int holders = 0, last = -1;
            for (int i = lane; i < p.B; i += 32)
                if (s_page[i] == page) {
                    ++holders;
                    last = i;
                }
            holders = __reduce_add_sync(~0u, holders);
            last = __reduce_max_sync(~0u, last);
            copy = !(holders >= p.refs_in[page] && last == b);
        }
        if (lane == 0) flag[b] = copy;
    }
    cluster_sync();

    // pages and copies before each row: packed sums, 1024 rows at a time (a
    // row may ask for 2^26 pages, so that all of them together pass 32 bits)
    static_assert(AQ_CACHE_MAX_ROWS < 1 << kCopyBits, "copies fit below the pages");
    constexpr long long kCopyMask = (1 << kCopyBits) - 1;
    long long carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        long long mine = 0;
        if (b < p.B && !s_bad) {
            const int len = p.lens_in[b], copy = __ldcg(flag + b);
            const int need =
                pages_of(len + p.arg0[b], p.page_log2) - pages_of(len, p.page_log2) + copy;
            mine = ((long long)need << kCopyBits) | copy;
        }
        long long before = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(~0u, before, o);
            if (lane >= o) before += v;
        }
        if (lane == 31) s_scan[warp] = before;
        __syncthreads();
        long long skip = carry, all = carry;
        for (int w = 0; w < kWarps; ++w) {
            const long long v = s_scan[w];
            if (w < warp) skip += v;
            all += v;
        }
        carry = all;
        if (b < p.B) {
            // (more than an int's worth are more than the pool has: not used then)
            s_base[b] = (int)((skip + before - mine) >> kCopyBits);
            // copies before this row, or -1 - that where it has none itself
            const int c = (int)((skip + before - mine) & kCopyMask);
            s_copy[b] = (mine & 1) ? c : -1 - c;
        }
        __syncthreads();
    }
    const long long need = carry >> kCopyBits;
    const int copies = (int)(carry & kCopyMask);
    int total = 0, rank0 = 0;
    for (int r = 0; r < kCtas; ++r) {
        if (r < rank) rank0 += s_free[r];
        total += s_free[r];
    }
    const bool none = s_bad != 0 || need > total;
    if (!none) {
        // the run's free pages, by rank
        int at = rank0 + s_warp[warp];
        for (int64_t i = run.begin; i < run.end && at < need; i += 32) {
            const bool is_free = i + lane < run.end && p.refs_in[i + lane] <= 0;
            const unsigned m = __ballot_sync(~0u, is_free);
            const int r = at + __popc(m & ((1u << lane) - 1u));
            at += __popc(m);
            if (!is_free || r >= need) continue;
            int lo = 0, hi = p.B;  // the last row with s_base <= r
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_base[mid] <= r)
                    lo = mid;
                else
                    hi = mid;
            }
            const int len = p.lens_in[lo], c = s_copy[lo];
            int j = r - s_base[lo], spot;
            if (c >= 0 && j == 0) {
                spot = len >> p.page_log2;
                list[3 * c] = s_page[lo];
                list[3 * c + 1] = (int)(i + lane);
                list[3 * c + 2] = len & mask;
            } else {
                spot = pages_of(len, p.page_log2) + j - (c >= 0);
            }
            p.table[(int64_t)lo * p.max_pages + spot] = (int)(i + lane);
            p.refs[i + lane] = 1;
        }
    }
    cluster_sync();
    if (!none && rank == 0)
        for (int b = threadIdx.x; b < p.B; b += kThreads) {
            if (s_copy[b] >= 0) atomicSub(&p.refs[s_page[b]], 1);
            p.lens[b] = p.lens_in[b] + p.arg0[b];
        }
    if (outside && !none) atomicMax(&p.status[0], 3);
    if (rank == 0 && threadIdx.x == 0) {
        if (none) atomicMax(&p.status[0], s_bad ? 2 : 1);
        p.status[1] = s_bad ? s_bad : none ? (int)min(need - total, (long long)INT32_MAX) : 0;
        p.status[2] = none ? 0 : (int)need;
        p.status[3] = none ? 0 : copies;
        p.ws[0] = none ? 0 : copies;
    }
}

// Compact: with n live pages, the live pages at n and above move to the free
// ones below it, the last live page to the first of them; counts and the
// tables' entries follow (the pages by copy_pages_kernel).  status[2] live
// pages, status[3] pages moved.
//
// ws: [0] number of moves, then sources [n_pages], targets [n_pages] and, by
// page, its move [n_pages].
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads) compact_kernel(
    const TableParams p) {
    __shared__ int s_live[kCtas], s_warp[kWarps], s_holes, s_all[kCtas], s_bad;
    const int rank = (int)cluster_ctarank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) s_holes = s_bad = 0;
    __syncthreads();
    cluster_sync();
    launch_dependents();
    grid_dependency_wait();
    if (p.refs != p.refs_in)
        for (int64_t i = (int64_t)rank * kThreads + threadIdx.x; i < p.n_pages;
             i += (int64_t)kCtas * kThreads)
            p.refs[i] = p.refs_in[i];
    if (rank == 0 && threadIdx.x < 4) p.status[threadIdx.x] = 0;
    int32_t *src = p.ws + 1, *dst = src + p.n_pages, *map = dst + p.n_pages;

    const Run run = warp_run(p, rank);
    const int live = count_live(p.refs_in, run);
    if (lane == 0) s_warp[warp] = live;
    int bad = 0;
    for (int b = threadIdx.x; b < p.B; b += kThreads) bad += !sound_len(p, p.lens_in[b]);
    if (bad) atomicAdd(&s_bad, bad);
    __syncthreads();
    if (warp == 0) {
        int n = s_warp[lane], before = n;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(~0u, before, o);
            if (lane >= o) before += v;
        }
        s_warp[lane] = before - n;
        if (lane == 31) publish(s_live, rank, before);
    }
    cluster_sync();
    int64_t count = 0;
    int at = s_warp[warp];
    for (int r = 0; r < kCtas; ++r) {
        if (r < rank) at += s_live[r];
        count += s_live[r];
    }
    const bool none = s_bad != 0;
    int holes = 0;
    if (!none)
        for (int64_t i = run.begin; i < run.end; i += 32) {
            const int64_t me = i + lane;
            const bool in = me < run.end, is_live = in && p.refs_in[me] > 0;
            const unsigned m = __ballot_sync(~0u, is_live);
            const int before = at + __popc(m & ((1u << lane) - 1u));
            at += __popc(m);
            if (in && !is_live && me < count) {
                dst[me - before] = (int)me;
                ++holes;
            }
            if (is_live && me >= count) src[count - 1 - before] = (int)me;
            if (in && me >= count) map[me] = is_live ? (int)(count - 1 - before) : -1;
        }
    holes = __reduce_add_sync(~0u, holes);
    if (lane == 0 && holes) atomicAdd(&s_holes, holes);
    __syncthreads();
    if (threadIdx.x == 0) publish(s_all, rank, s_holes);
    cluster_sync();
    int moves = 0;
    for (int r = 0; r < kCtas; ++r) moves += s_all[r];
    // counts: a move's source and target belong to no other move
    for (int64_t k = (int64_t)rank * kThreads + threadIdx.x; k < moves;
         k += (int64_t)kCtas * kThreads) {
        const int from = __ldcg(src + k), to = __ldcg(dst + k);
        p.refs[to] = p.refs_in[from];
        p.refs[from] = 0;
    }
    const int64_t entries = (int64_t)p.B * p.max_pages;
    for (int64_t i = (int64_t)rank * kThreads + threadIdx.x; i < entries;
         i += (int64_t)kCtas * kThreads) {
        const int b = (int)(i / p.max_pages), spot = (int)(i - (int64_t)b * p.max_pages);
        int id = p.table_in[i];
        if (!none && spot < pages_of(p.lens_in[b], p.page_log2)) {
            if (id < 0 || id >= p.n_pages)
                atomicMax(&p.status[0], 3);
            else if (id >= count) {
                const int k = __ldcg(map + id);
                if (k >= 0)
                    id = __ldcg(dst + k);
                else
                    atomicMax(&p.status[0], 3);  // an entry that names a free page
            }
        }
        if (p.table != p.table_in || id != p.table_in[i]) p.table[i] = id;
    }
    if (rank == 0 && threadIdx.x == 0) {
        if (none) atomicMax(&p.status[0], 2);
        p.status[1] = s_bad;
        p.status[2] = none ? 0 : (int)count;
        p.status[3] = moves;
        p.ws[0] = moves;
    }
}

// ---------------------------------------------------------------------------
// Copies of pages.
// ---------------------------------------------------------------------------

struct CopyParams {
    uint8_t *pool;
    const int32_t *src, *dst;  // copy_pages
    const int32_t *list;       // copy_rows: (source, target, rows) each
    const int32_t *count;      // on the device, or null: n
    int64_t n;
    int64_t layers;
    CacheGeom c;
    uint32_t *err;
};

constexpr int kCopyThreads = 256;
constexpr int kCopyChunk = kCopyThreads * 16 * 4;  // bytes a CTA copies at a time

// Whole pages: units of 16 KB, four 16-byte loads a thread in flight.  2000
// pages of two layers, 580 MB in and out, take 85 us: the copy rate of the
// device (6.8 TB/s).
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const CopyParams p) {
    launch_dependents();
    grid_dependency_wait();
    const int64_t n = p.count ? *p.count : p.n;
    const int64_t chunks = (p.c.page_bytes + kCopyChunk - 1) / kCopyChunk;
    const int64_t units = n * p.layers * chunks;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t k = u / (p.layers * chunks), rest = u - k * p.layers * chunks;
        const int64_t layer = rest / chunks, chunk = rest - layer * chunks;
        const int64_t s = p.src[k], d = p.dst[k];
        if (s < 0 || s >= p.c.n_pages || d < 0 || d >= p.c.n_pages) {
            if (threadIdx.x == 0 && rest == 0) atomicOr(p.err, ERR_CACHE_TABLE);
            continue;
        }
        if (s == d) continue;
        uint8_t *base = p.pool + layer * p.c.n_pages * p.c.page_bytes;
        const uint4 *from = reinterpret_cast<const uint4 *>(base + s * p.c.page_bytes);
        uint4 *to = reinterpret_cast<uint4 *>(base + d * p.c.page_bytes);
        const int64_t at = chunk * (kCopyChunk / 16) + threadIdx.x, end = p.c.page_bytes / 16;
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at + j * kCopyThreads < end) v[j] = from[at + j * kCopyThreads];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at + j * kCopyThreads < end) to[at + j * kCopyThreads] = v[j];
    }
}

// The first rows of pages: the four parts of each (layer, head) record, a
// warp a record with eight loads a lane under way (a CTA a record, one load a
// thread, took 19.4 us for 256 pages of four layers, this 13.8; the bytes are
// 11.0).
__global__ void __launch_bounds__(kCopyThreads) copy_rows_kernel(const CopyParams p) {
    launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t each = p.layers * p.c.KV, units = *p.count * each;
    const int64_t warps = (int64_t)gridDim.x * (kCopyThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); u < units;
         u += warps) {
        const int64_t k = u / each, rest = u - k * each;
        const int64_t layer = rest / p.c.KV, kv = rest - layer * p.c.KV;
        const int64_t s = p.list[3 * k], d = p.list[3 * k + 1];
        const int rows = p.list[3 * k + 2];
        uint8_t *base = p.pool + layer * p.c.n_pages * p.c.page_bytes + kv * p.c.rec;
        const uint8_t *from = base + s * p.c.page_bytes;
        uint8_t *to = base + d * p.c.page_bytes;
        // codes: 16-byte pieces of K, then of V (a row is 32 bytes or more);
        // (scale, bias) pairs: 4-byte words
        const int cw = rows * p.c.rb / 16, sw = rows * p.c.groups;
        auto code_at = [&](int i) { return (i < cw ? 0 : p.c.side_codes) + 16 * (i < cw ? i : i - cw); };
        auto pair_at = [&](int i) {
            return 2 * p.c.side_codes + (i < sw ? 0 : p.c.side_sb) + 4 * (i < sw ? i : i - sw);
        };
        for (int i0 = lane; i0 < 2 * cw; i0 += 256) {
            uint4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i0 + 32 * j < 2 * cw)
                    v[j] = *reinterpret_cast<const uint4 *>(from + code_at(i0 + 32 * j));
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i0 + 32 * j < 2 * cw)
                    *reinterpret_cast<uint4 *>(to + code_at(i0 + 32 * j)) = v[j];
        }
        for (int i0 = lane; i0 < 2 * sw; i0 += 128) {
            uint32_t v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + 32 * j < 2 * sw)
                    v[j] = *reinterpret_cast<const uint32_t *>(from + pair_at(i0 + 32 * j));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + 32 * j < 2 * sw)
                    *reinterpret_cast<uint32_t *>(to + pair_at(i0 + 32 * j)) = v[j];
        }
    }
}

template <class P>
cudaError_t launch_pdl(void (*kern)(P), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                       const P &prm) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, prm);
}

// The error word of the current device, looked up once a device.
cudaError_t error_word(uint32_t **err) {
    return device_symbol(g_cache_error, err);
}

TableParams table_params(const CacheTables &t, const aq_cache *c) {
    TableParams p = {};
    const CacheGeom g = cache_geom(c);
    p.refs_in = t.refs_in;
    p.table_in = t.table_in;
    p.lens_in = t.lens_in;
    p.refs = t.refs;
    p.table = t.table;
    p.lens = t.lens;
    p.arg0 = t.arg0;
    p.arg1 = t.arg1;
    p.status = t.status;
    p.ws = t.ws;
    p.n_pages = c->n_pages;
    p.max_pages = t.max_pages;
    p.B = (int)t.B;
    p.page = c->page;
    p.page_log2 = g.page_log2;
    return p;
}

CopyParams copy_params(const aq_cache *c) {
    CopyParams p = {};
    p.pool = static_cast<uint8_t *>(c->pool_dev);
    p.layers = c->layers;
    p.c = cache_geom(c);
    return p;
}

}  // namespace

cudaError_t cache_append_launch(const aq_cache *c, int64_t layer, int dtype, const void *k,
                                int64_t k_stride, const void *v, int64_t v_stride, void *k_out,
                                void *v_out, int64_t T, const int32_t *cu, const int32_t *start,
                                const int32_t *table, int64_t B, int64_t max_pages,
                                cudaStream_t stream) {
    RowParams p = {};
    p.c = cache_geom(c);
    p.layer = static_cast<uint8_t *>(c->pool_dev) + layer * c->n_pages * p.c.page_bytes;
    p.in[0] = k;
    p.in[1] = v;
    p.in_stride[0] = k_stride;
    p.in_stride[1] = v_stride;
    p.out[0] = k_out;
    p.out[1] = v_out;
    p.cu = cu;
    p.start = start;
    p.table = table;
    p.T = T;
    p.B = (int)B;
    p.max_pages = max_pages;
    const cudaError_t e = error_word(&p.err);
    if (e != cudaSuccess) return e;
    const int per_token = p.c.KV * p.c.D / 8;
    while (8 << p.head_log2 < p.c.D) ++p.head_log2;
    while (8 << p.lane_log2 < p.c.group) ++p.lane_log2;
    p.span = 32;
    while (per_token % p.span != 0) p.span /= 2;
    // The chain of loads that finds a page takes longer than a token's data:
    // where there are tokens enough to fill the device, a lane group takes two
    // and looks both up at once (append and read, 8 heads of 128, 16k tokens:
    // 57.7 us with one, 53.3 with two, 53.8 with four; 2k: 12.0, 13.2, 17.2)
    p.each = T >= 4096 ? 2 : 1;
    const int64_t tokens = (int64_t)(kRowThreads / p.span) * p.each;  // a CTA
    const dim3 grid((unsigned)((T + tokens - 1) / tokens), 2, 1);
    void (*kern)(RowParams);
    const bool bf = dtype == AQ_BF16;
    if (k)
        kern = c->bits == 4 ? (bf ? append_kernel<4, true> : append_kernel<4, false>)
                            : (bf ? append_kernel<8, true> : append_kernel<8, false>);
    else
        kern = c->bits == 4 ? (bf ? read_kernel<4, true> : read_kernel<4, false>)
                            : (bf ? read_kernel<8, true> : read_kernel<8, false>);
    kern<<<grid, kRowThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t cache_fork_launch(const aq_cache *c, const CacheTables &t, cudaStream_t stream) {
    return launch_pdl(fork_kernel, dim3(kCtas), kThreads, 0, stream, table_params(t, c));
}

cudaError_t cache_trim_launch(const aq_cache *c, const CacheTables &t, cudaStream_t stream) {
    return launch_pdl(trim_kernel, dim3(kCtas), kThreads, 0, stream, table_params(t, c));
}

cudaError_t cache_grow_launch(const aq_cache *c, const CacheTables &t, cudaStream_t stream) {
    const size_t smem = 3 * sizeof(int) * (size_t)t.B;
    static const cudaError_t attr =
        cudaFuncSetAttribute(grow_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             3 * (int)sizeof(int) * AQ_CACHE_MAX_ROWS);
    if (attr != cudaSuccess) return attr;
    cudaError_t e =
        launch_pdl(grow_kernel, dim3(kCtas), kThreads, smem, stream, table_params(t, c));
    if (e != cudaSuccess) return e;
    CopyParams p = copy_params(c);
    p.list = t.ws + 1;
    p.count = t.ws;
    return launch_pdl(copy_rows_kernel, dim3((unsigned)(8 * num_sms())), kCopyThreads, 0, stream,
                      p);
}

cudaError_t cache_compact_launch(const aq_cache *c, const CacheTables &t, cudaStream_t stream) {
    cudaError_t e =
        launch_pdl(compact_kernel, dim3(kCtas), kThreads, 0, stream, table_params(t, c));
    if (e != cudaSuccess) return e;
    CopyParams p = copy_params(c);
    p.src = t.ws + 1;
    p.dst = t.ws + 1 + c->n_pages;
    p.count = t.ws;
    e = error_word(&p.err);
    if (e != cudaSuccess) return e;
    return launch_pdl(copy_pages_kernel, dim3((unsigned)(8 * num_sms())), kCopyThreads, 0, stream,
                      p);
}

cudaError_t cache_copy_launch(const aq_cache *c, const int32_t *src, const int32_t *dst, int64_t n,
                              cudaStream_t stream) {
    CopyParams p = copy_params(c);
    p.src = src;
    p.dst = dst;
    p.n = n;
    const cudaError_t e = error_word(&p.err);
    if (e != cudaSuccess) return e;
    return launch_pdl(copy_pages_kernel, dim3((unsigned)(8 * num_sms())), kCopyThreads, 0, stream,
                      p);
}

cudaError_t cache_read_error(uint32_t *code, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_cache_error, sizeof(uint32_t));
    if (e != cudaSuccess || !clear) return e;
    const uint32_t zero = 0;
    return cudaMemcpyToSymbol(g_cache_error, &zero, sizeof(uint32_t));
}

}  // namespace aq
