// The mixture-of-experts layer's router, its sum over a token's experts, and
// the host side of both and of the experts' products (aq_moe.cuh).
//
// Router: logits l[t][e] = x[t] . Wr[e], a score p = softmax(l[t]) or
// 1 / (1 + exp(-l)), the top_k largest l (with a bias: the largest p + bias),
// ties to the lowest index, weights p / (sum of the chosen p) or p, times a
// factor.  The choice is that of exact arithmetic as far as 64 bits tell:
//   * the logits are fp32 sums of MMA steps with the additions' rounding errors
//     carried along, beside them the sums of |x w|, which bound what the steps
//     truncate;
//   * experts whose value is farther from the k-th largest than the bounds
//     are in or out for certain; where others are left to choose from, their
//     logits are summed again with the rounding errors carried along (products
//     of two 16-bit floats are exact in fp32, two-sums keep what each addition
//     rounds off), which is good to about 2^-46 of the sum of |x w|, or in 64
//     bits where a product or a sum passes fp32's range at either end.
//   * weights come from the fp32 logits.
// One launch, bound by latency (loads, two cluster barriers, the choice): one
// token and 128 experts of 2048 6 us; 256 experts of 5120 11 us for one token, 21
// for 65 to 128, 31 for 256 (eight warps an SM, which wait for loads 43 % of the
// time; L2 is 4 % busy).  The bound that the sums' rounding errors allow leaves
// about one of 300 tokens of the last case to be summed again; without them it
// was one of 25.  A call with one such token takes 36 us instead of 31, with
// three 40, since one warp sums for its token.
// A cluster of 8 or 16 CTAs takes 8 or 16 tokens: its CTAs slice K, their warps deal
// the experts (16 an MMA tile) and, where there are fewer tiles than warps,
// slice K further; the parts are sent to the CTA that chooses for the token,
// one warp a token.
#include "aq_device.h"
#include "aq_moe.h"
#include "aq_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <initializer_list>

namespace aq {
namespace {

constexpr int kOwners = 8;  // CTAs of a cluster that choose, for every eighth token each
constexpr int kWarps = 8;
constexpr int kThreads = 256;

struct RouteParams {
    const uint16_t *x, *w;
    const float *bias;
    int32_t *ids;
    float *weights;
    int T, E, K, top, score, normalize;
    float scale;
    int cluster;  // CTAs of a cluster, 8 or 16
    int slices;   // of K: one a CTA of the cluster, more where there are fewer tiles than warps
};

template <bool BF16>
__device__ __forceinline__ void mma_x(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool BF16>
__device__ __forceinline__ float value(uint16_t bits) {
    if constexpr (BF16)
        return __uint_as_float((uint32_t)bits << 16);
    else
        return __half2float(__ushort_as_half(bits));
}

// s + e = s + v exactly, what the addition rounds off added to e.
__device__ __forceinline__ void two_sum(float &s, float &e, float v) {
    const float t = __fadd_rn(s, v);
    const float b = __fsub_rn(t, s);
    e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(v, b)));
    s = t;
}

// One logit in 64 bits, in every lane: finite for every finite row.
template <bool BF16>
__device__ __noinline__ double wide_logit(const uint16_t *x, const uint16_t *w, int K) {
    double d = 0.0;
    for (int k = (threadIdx.x & 31) * 8; k < K; k += 256)
#pragma unroll
        for (int i = 0; i < 8; ++i) d = fma((double)value<BF16>(x[k + i]), (double)value<BF16>(w[k + i]), d);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
    return d;
}

// One logit to about 2^-46 of its sum of magnitudes, in every lane.  Four sums
// a lane, so that the additions of one do not wait for another's.  tiny: that
// sum is so small that what products below 2^-126 lose counts.
template <bool BF16>
__device__ __noinline__ double precise_logit(const uint16_t *x, const uint16_t *w, int K, bool tiny) {
    if (tiny) return wide_logit<BF16>(x, w, K);
    const int lane = threadIdx.x & 31;
    float s[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int k = lane * 8; k < K; k += 256) {
        const uint4 a = *reinterpret_cast<const uint4 *>(x + k), b = *reinterpret_cast<const uint4 *>(w + k);
        const uint32_t xa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            two_sum(s[i], e[i], __fmul_rn(value<BF16>((uint16_t)xa[i]), value<BF16>((uint16_t)wb[i])));
            two_sum(s[i], e[i], __fmul_rn(value<BF16>((uint16_t)(xa[i] >> 16)), value<BF16>((uint16_t)(wb[i] >> 16))));
        }
    }
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) d += (double)s[i] + (double)e[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
    // (a sum that passes the largest float, though the logit may not, ends as NaN)
    return fabs(d) < INFINITY ? d : wide_logit<BF16>(x, w, K);
}

// What a row of x holds, in every lane.
enum Row { ROW_ZEROS, ROW_FINITE, ROW_OTHER };  // zeros alone; finite numbers; infinities or NaN too
template <bool BF16>
__device__ Row row_holds(const uint16_t *x, int K) {
    constexpr uint32_t kExp = BF16 ? 0x7F80u : 0x7C00u;
    bool finite = true;
    uint32_t any = 0u;
    for (int k = (threadIdx.x & 31) * 8; k < K; k += 256) {
        const uint4 a = *reinterpret_cast<const uint4 *>(x + k);
        const uint32_t v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            finite = finite && (v[i] & kExp) != kExp && (v[i] >> 16 & kExp) != kExp;
            any |= v[i] & 0x7FFF7FFFu;
        }
    }
    if (!__all_sync(0xFFFFFFFFu, finite)) return ROW_OTHER;
    return __any_sync(0xFFFFFFFFu, any != 0u) ? ROW_FINITE : ROW_ZEROS;
}

// Floats in the order of unsigned integers; NaN below everything.
__device__ __forceinline__ uint32_t ordered(float v) {
    if (!(v == v)) return 0u;
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The choice for token t by one warp, of up to 32 LANES experts.  sums: [2][E],
// logits and their sums of magnitudes; keep: E doubles for values summed again.
template <bool BF16, int LANES>
__device__ void choose(const RouteParams &p, int t, const float *sums, double *keep) {
    const int lane = threadIdx.x & 31;
    const int per = (p.E + 31) / 32;
    const bool sigmoid = p.score == AQ_SCORE_SIGMOID;
    float logit[LANES], val[LANES];
    float slack = 0.f;      // the largest error bound of a value
    bool lost = false;      // an expert's sums pass fp32's range: they tell nothing
    uint32_t open = 0u;     // experts not yet taken, by position
    // what the sums leave out: a product of 16 may truncate each of its 16 terms
    // at 2^-24 of the largest, 4 * 2^-22 of the magnitudes at most (the most seen,
    // with one term 2^23 to 2^27 times the others, is 1.5 * 2^-22); the last
    // rounding is 2^-24 of the logit, what the errors' own sums and those of the
    // magnitudes round is smaller by 2^-20.  Products and sums below 2^-126 may
    // count as zeros.
    constexpr float kUlps = 4.5f * 2.384185791015625e-07f;
    const float least = (float)p.K * 1.175494350822287508e-38f;
#pragma unroll
    for (int j = 0; j < LANES; ++j) {
        logit[j] = val[j] = -INFINITY;
        const int e = j * 32 + lane;
        if (j < per && e < p.E) {
            const float s = sums[e];
            logit[j] = s;
            float bound = fmaf(kUlps, sums[p.E + e], least);
            lost = lost || !(bound < INFINITY);
            float v = s;
            if (p.bias) {
                v = 1.f / (1.f + expf(-s)) + p.bias[e];
                bound = 0.25f * bound + 4.76837158203125e-07f * (1.f + fabsf(v));
            }
            val[j] = v == v ? v : -INFINITY;
            if (bound < INFINITY) slack = fmaxf(slack, bound);
            open |= 1u << j;
        }
    }
    slack = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(slack)));
    lost = __any_sync(0xFFFFFFFFu, lost);

    // the top_k of the fp32 values: the last one taken is the border
    uint32_t left = open, taken = 0u;
    float border = 0.f;
    for (int n = 0; n < p.top; ++n) {
        uint32_t best = 0u;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int j = 0; j < LANES; ++j) {
            const uint32_t o = ordered(val[j]);
            if ((left >> j & 1u) && (at == 0x7FFFFFFF || o > best)) {
                best = o;
                at = j * 32 + lane;
            }
        }
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
        const int e = __reduce_min_sync(0xFFFFFFFFu, best == top ? at : 0x7FFFFFFF);
        if (at == e) {
            left &= ~(1u << (e >> 5));
            taken |= 1u << (e >> 5);
        }
        border = top & 0x80000000u ? __uint_as_float(top & 0x7FFFFFFFu) : __uint_as_float(~top);
    }
    // the k-th largest exact value lies within slack of the border
    uint32_t sure = 0u, doubt = 0u;
#pragma unroll
    for (int j = 0; j < LANES; ++j) {
        if (!(open >> j & 1u)) continue;
        if (val[j] > border + 2.f * slack)
            sure |= 1u << j;
        else if (val[j] >= border - 2.f * slack)
            doubt |= 1u << j;
    }
    if (lost) {  // the border is nowhere
        sure = 0u;
        doubt = open;
    }
    const int n_sure = __reduce_add_sync(0xFFFFFFFFu, __popc(sure));
    const int n_doubt = __reduce_add_sync(0xFFFFFFFFu, __popc(doubt));
    const uint16_t *x = p.x + (size_t)t * p.K;
    // (the fp32 choice stands where the border is a bias that is not finite)
    bool again = lost || (n_sure + n_doubt > p.top && fabsf(border) < INFINITY);
    bool zeros = false;
    if (again) {
        // An empty slot of a padded batch, zeros or whatever was there, is not worth
        // E sums: the fp32 choice stands for a token that is not finite, and for
        // zeros, whose logits are exact, as far as there are no biases to add.
        bool some = false;
#pragma unroll
        for (int j = 0; j < LANES; ++j) some = some || ((open >> j & 1u) && sums[p.E + j * 32 + lane] != 0.f);
        if (lost || !__any_sync(0xFFFFFFFFu, some)) {
            const Row row = row_holds<BF16>(x, p.K);
            zeros = row == ROW_ZEROS && !lost;  // (infinite weights times zero are NaN)
            again = row != ROW_OTHER && !(zeros && !p.bias);
        }
    }
    if (again) {
#pragma unroll
        for (int j = 0; j < LANES; ++j) {
            if (zeros) {
                const int e = j * 32 + lane;
                if (doubt >> j & 1u) keep[e] = 0.5 + (double)p.bias[e];
                continue;
            }
            for (uint32_t m = __ballot_sync(0xFFFFFFFFu, doubt >> j & 1u); m; m &= m - 1u) {
                const int e = j * 32 + __ffs(m) - 1;
                const bool tiny = !(sums[p.E + e] > 67108864.f * least);  // 2^-46 of more is above what is lost
                const double d = precise_logit<BF16>(x, p.w + (size_t)e * p.K, p.K, tiny);
                if (lane == (e & 31)) {
                    const double v = p.bias ? 1.0 / (1.0 + exp(-d)) + (double)p.bias[e] : d;
                    keep[e] = v == v ? v : -INFINITY;  // (the lanes below agree on an order without NaN)
                    if (lost) logit[j] = (float)d;
                }
            }
        }
        __syncwarp();
        taken = sure;
        for (int n = n_sure; n < p.top; ++n) {
            double best = 0.0;
            int at = 0x7FFFFFFF;
            for (uint32_t m = doubt; m; m &= m - 1u) {
                const int e = (__ffs(m) - 1) * 32 + lane;
                if (at == 0x7FFFFFFF || keep[e] > best) {
                    best = keep[e];
                    at = e;
                }
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double b = __shfl_xor_sync(0xFFFFFFFFu, best, o);
                const int a = __shfl_xor_sync(0xFFFFFFFFu, at, o);
                if (a != 0x7FFFFFFF &&
                    (at == 0x7FFFFFFF || b > best || (b == best && a < at))) {
                    best = b;
                    at = a;
                }
            }
            if (lane == (at & 31)) {
                doubt &= ~(1u << (at >> 5));
                taken |= 1u << (at >> 5);
            }
        }
    }

    // weights: with m the largest (chosen) logit, exp(l - m); sigmoids times
    // exp(-min(m, 0)), so that a sum of tiny ones does not vanish
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < LANES; ++j)
        if ((sigmoid || p.normalize ? taken : open) >> j & 1u) m = fmaxf(m, logit[j]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (sigmoid) m = p.normalize ? fminf(m, 0.f) : 0.f;
    float sum = 0.f;
    const uint32_t over = p.normalize ? taken : open;
#pragma unroll
    for (int j = 0; j < LANES; ++j) {
        // sigmoid: exp(-m) / (1 + exp(-l)), for l < 0 as exp(l - m) / (1 + exp(l))
        const float l = logit[j];
        val[j] = !sigmoid ? expf(l - m)
                 : l < 0.f ? expf(l - m) / (1.f + expf(l))
                           : expf(-m) / (1.f + expf(-l));
        if (over >> j & 1u) sum += val[j];
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (sigmoid && !p.normalize) sum = 1.f;
    int before = 0;
#pragma unroll
    for (int j = 0; j < LANES; ++j) {
        const uint32_t on = __ballot_sync(0xFFFFFFFFu, taken >> j & 1u);
        const int place = before + __popc(on & ((1u << lane) - 1u));
        if ((taken >> j & 1u) && place < p.top) {
            const size_t at = (size_t)t * p.top + place;
            p.ids[at] = j * 32 + lane;
            p.weights[at] = val[j] / sum * p.scale;
        }
        before += __popc(on);
    }
}

template <bool BF16, int NB, int LANES>
__global__ void __launch_bounds__(kThreads) route_kernel(const __grid_constant__ RouteParams p) {
    constexpr int TOKENS = 8 * NB, MINE = TOKENS / kOwners;  // a CTA chooses for MINE tokens
    extern __shared__ __align__(16) uint8_t dyn[];
    // [MINE][slices][3][E] parts from all CTAs, [MINE][E] doubles
    float *parts = reinterpret_cast<float *>(dyn);
    double *keep = reinterpret_cast<double *>(dyn + ((MINE * p.slices * 3 * p.E * 4 + 15) & ~15));
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0);
    const int rank = (int)cluster_ctarank();
    const int t0 = (int)blockIdx.x / p.cluster * TOKENS;
    launch_dependents();
    cluster_sync();  // every CTA of the cluster runs before its shared memory is written
    grid_dependency_wait();

    // A warp takes tiles warp / cuts, + kWarps / cuts, .. over one slice of K, in
    // steps of 32 values: lane (g, q) reads 8 of them of rows g and g + 8, and of
    // token g of each block of 8.
    const int cuts = p.slices / p.cluster, slice = rank * cuts + warp % cuts;
    const int steps = p.K / 32;
    const int k_beg = (int)((int64_t)steps * slice / p.slices);
    const int k_end = (int)((int64_t)steps * (slice + 1) / p.slices);
    const uint16_t *xs[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) xs[nb] = p.x + (size_t)min(t0 + nb * 8 + g, p.T - 1) * p.K + 8 * q;
    for (int tile = warp / cuts; tile * 16 < p.E; tile += kWarps / cuts) {
        const int ra = min(tile * 16 + g, p.E - 1), rb = min(tile * 16 + 8 + g, p.E - 1);
        const uint16_t *wa = p.w + (size_t)ra * p.K + 8 * q, *wb = p.w + (size_t)rb * p.K + 8 * q;
        // each product starts from zero and is added with the rounding error: s + r;
        // m the sums of magnitudes
        float s[NB][4], r[NB][4], m[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nb][i] = r[nb][i] = m[nb][i] = 0.f;
#pragma unroll(NB == 1 ? 8 : 4)
        for (int k = k_beg; k < k_end; ++k) {
            const uint4 a = *reinterpret_cast<const uint4 *>(wa + 32 * k);
            const uint4 b = *reinterpret_cast<const uint4 *>(wb + 32 * k);
            constexpr uint32_t kAbs = 0x7FFF7FFFu;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const uint4 x = *reinterpret_cast<const uint4 *>(xs[nb] + 32 * k);
                float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
                mma_x<BF16>(d0, a.x, b.x, a.y, b.y, x.x, x.y);
                mma_x<BF16>(d1, a.z, b.z, a.w, b.w, x.z, x.w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    two_sum(s[nb][i], r[nb][i], d0[i]);
                    two_sum(s[nb][i], r[nb][i], d1[i]);
                }
                mma_x<BF16>(m[nb], a.x & kAbs, b.x & kAbs, a.y & kAbs, b.y & kAbs, x.x & kAbs,
                            x.y & kAbs);
                mma_x<BF16>(m[nb], a.z & kAbs, b.z & kAbs, a.w & kAbs, b.w & kAbs, x.z & kAbs,
                            x.w & kAbs);
            }
        }
        // to the tokens' CTAs
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = tile * 16 + g + 8 * (j >> 1), n = nb * 8 + 2 * q + (j & 1);
                if (e >= p.E || t0 + n >= p.T) continue;
                const float *to = parts + ((size_t)(n / kOwners) * p.slices + slice) * 3 * p.E + e;
                const uint32_t at = map_to_rank(smem_u32(to), (uint32_t)(n % kOwners));
                st_dsmem_f32(at, s[nb][j]);
                st_dsmem_f32(at + 4u * (uint32_t)p.E, r[nb][j]);
                st_dsmem_f32(at + 8u * (uint32_t)p.E, m[nb][j]);
            }
    }
    cluster_sync();
    if (rank >= kOwners) return;
    // the slices' parts, in order, into the first slice's place
    for (int i = threadIdx.x; i < MINE * p.E; i += kThreads) {
        const int n = i / p.E;
        float *from = parts + (size_t)n * p.slices * 3 * p.E + (i - n * p.E);
        float s = 0.f, r = 0.f, m = 0.f;
#pragma unroll 4
        for (int k = 0; k < p.slices; ++k) {
            const float *f = from + (size_t)k * 3 * p.E;
            two_sum(s, r, f[0]);
            r += f[p.E];
            m += f[2 * p.E];
        }
        from[0] = s + r;
        from[p.E] = m;
    }
    __syncthreads();
    if (warp < MINE) {
        const int t = t0 + warp * kOwners + rank;
        if (t < p.T) choose<BF16, LANES>(p, t, parts + (size_t)warp * p.slices * 3 * p.E, keep + (size_t)warp * p.E);
    }
}

// y[t] = sum over j of weight * d[t * top + j], entries without an expert left
// out, in j's order; four columns a thread.
struct CombineParams {
    const int32_t *ids;
    const float *weights, *parts;
    void *out;
    int T, top, E, H, dtype;
};

__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ CombineParams p) {
    launch_dependents();
    grid_dependency_wait();
    const int per = p.H / 4;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (int64_t)p.T * per) return;
    const int t = (int)(i / per), c = (int)(i - (int64_t)t * per);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < p.top; ++j) {
        const int64_t at = (int64_t)t * p.top + j;
        const int e = p.ids[at];
        if (e < 0 || e >= p.E) continue;
        const float w = p.weights[at];
        const float4 v = reinterpret_cast<const float4 *>(p.parts)[at * per + c];
        s.x = fmaf(w, v.x, s.x);
        s.y = fmaf(w, v.y, s.y);
        s.z = fmaf(w, v.z, s.z);
        s.w = fmaf(w, v.w, s.w);
    }
    uint2 o;
    if (p.dtype == AQ_BF16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(s.x, s.y), b = __floats2bfloat162_rn(s.z, s.w);
        o = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
        o = make_uint2(pack_half2(s.x, s.y), pack_half2(s.z, s.w));
    }
    reinterpret_cast<uint2 *>(p.out)[i] = o;
}

template <bool BF16, int NB, int LANES>
cudaError_t route_run(RouteParams p, cudaStream_t stream) {
    auto *kern = route_kernel<BF16, NB, LANES>;
    // K in 16 slices where one cluster has much to read alone, if the device has
    // room for such a cluster; else in 8
    static PerDevice wide;
    p.cluster = 8;
    if (p.T <= 64 && (int64_t)p.E * p.K >= 1 << 19) {
        int dev = 0;
        const cudaError_t got = cudaGetDevice(&dev);
        if (got != cudaSuccess) return got;
        const bool w = wide(dev, [&] {
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(16);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = 112 * 1024;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 16;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
            if (e != cudaSuccess) cudaGetLastError();
            return e == cudaSuccess && n > 0;
        });
        if (w) p.cluster = 16;
    }
    p.slices = p.cluster * kWarps;
    for (int tiles = (p.E + 15) / 16, w = 1; w < tiles && w < kWarps; w *= 2) p.slices /= 2;
    const int mine = 8 * NB / kOwners;
    const size_t smem = (((size_t)mine * p.slices * 3 * p.E * 4 + 15) & ~(size_t)15) +
                        (size_t)mine * p.E * 8;
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e != cudaSuccess) return e;
    }
    const unsigned blocks = (unsigned)((p.T + 8 * NB - 1) / (8 * NB)) * (unsigned)p.cluster;
    return moe_launch(kern, dim3(blocks), kThreads, smem, p.cluster, stream, p);
}

// 8 tokens a cluster, or 16 for many, so that the weights are read half as often.
template <bool BF16>
cudaError_t route_sized(const RouteParams &p, cudaStream_t stream) {
    if (p.T > 64)
        return p.E <= 128   ? route_run<BF16, 2, 4>(p, stream)
               : p.E <= 256 ? route_run<BF16, 2, 8>(p, stream)
                            : route_run<BF16, 2, 16>(p, stream);
    return p.E <= 128   ? route_run<BF16, 1, 4>(p, stream)
           : p.E <= 256 ? route_run<BF16, 1, 8>(p, stream)
                        : route_run<BF16, 1, 16>(p, stream);
}

}  // namespace

cudaError_t moe_route_launch(const RouteArgs &a) {
    const aq_router &r = *a.router;
    RouteParams p = {};
    p.x = static_cast<const uint16_t *>(a.x);
    p.w = static_cast<const uint16_t *>(r.weight_dev);
    p.bias = r.bias_dev;
    p.ids = a.ids;
    p.weights = a.weights;
    p.T = (int)a.T;
    p.E = (int)r.E;
    p.K = (int)r.K;
    p.top = r.top_k;
    p.score = r.score;
    p.normalize = r.normalize;
    p.scale = r.scale;
    const bool bf16 = r.dtype == AQ_BF16;
    return bf16 ? route_sized<true>(p, a.stream) : route_sized<false>(p, a.stream);
}

namespace {
size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }
}  // namespace

// Which kernel runs a product over K, by the tokens a busy expert has on
// average, were all experts picked alike: 8, 16 or 32 columns at a time.
// Measured, us a layer's experts with 8 / 16 / 32 columns, packed, at 4 bits:
//   33 tokens, 6 of 64 experts of 5120 x 1536,   3.2 each  243 / 254 / 270
//   64 tokens, 6 of 64 experts of 2048 x 1024,   6.0 each  103 /  95 / 101
//   96 tokens, 6 of 64 experts of 5120 x 1536,   9.0 each  403 / 322 / 340
//   256 tokens, 8 of 128 experts of 2048 x 768,   16 each  496 / 367 / 316 (6 bits)
// and with at most 16 tokens, where an expert never has more than two blocks,
// 12 tokens on all of 4 experts of 4096 x 1536            61 /  44 /  46.
// The other widths choose alike (100 tokens, 6.3 each: 6 bits 231 / 189 / 204, 8
// bits 182 / 154 / 161; 64 tokens at 3 bits, 4.3 each: 124 / 113 / 127).  Whether
// the rows are packed first by a launch of their own, about 3 us, or by each CTA
// for itself, by the values a busy expert's tokens have (packed / not): 8 tokens
// of 8 experts of 4096, 9000 values, 205 / 228; 48 tokens of 64 experts of 2048,
// 6300, 82 / 83; one token of 2048, 32 / 28.
static int moe_variant(const aq_experts *x, int64_t T, int top, int64_t K) {
    const double E = (double)x->E;
    const double busy = top >= E ? E : E * (1.0 - std::pow(1.0 - top / E, (double)T));
    const double tokens = (double)T * top / busy;
    if (T <= 8 || tokens <= 4.0) return tokens * (double)K >= 8192.0 ? MOE_8_PACKED : MOE_8;
    return T <= 16 || tokens <= 10.0 ? MOE_16 : MOE_32;
}
static int up_variant(const aq_experts *x, int64_t T, int top) { return moe_variant(x, T, top, x->K); }
static int down_variant(const aq_experts *x, int64_t T, int top) { return moe_variant(x, T, top, x->inner); }

namespace {
struct Workspace {
    size_t h, parts, x, hp, bytes;  // offsets of h, the down products, the packed rows
};
Workspace workspace(const aq_experts *x, int64_t T, int top) {
    Workspace w;
    w.h = 0;
    w.parts = round256((size_t)T * top * x->inner * 4);
    w.x = w.parts + round256((size_t)T * top * x->K * 4);
    w.hp = w.x + (moe_packed(up_variant(x, T, top)) ? (size_t)moe_pack(T, x->K, x->group_size).bytes : 0);
    w.bytes = w.hp + (moe_packed(down_variant(x, T, top)) ? (size_t)moe_pack(T * top, x->inner, x->group_size).bytes : 0);
    return w;
}
}  // namespace

// h [T * top][I] and the down products [T * top][K], fp32, and packed rows.
size_t moe_workspace_bytes(const aq_experts *x, int64_t T, int top_k) {
    return workspace(x, T, top_k).bytes;
}

cudaError_t moe_experts_launch(const ExpertsArgs &a) {
    const aq_experts &x = *a.experts;
    const Workspace w = workspace(&x, a.T, a.top_k);
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    float *h = reinterpret_cast<float *>(ws), *parts = reinterpret_cast<float *>(ws + w.parts);
    typedef cudaError_t (*Product)(const MoeParams &, bool, int, cudaStream_t);
    typedef cudaError_t (*Pack)(const MoeParams &, bool, uint8_t *, cudaStream_t);
    const int at = x.bits == 8 ? 5 : x.bits - 2;
    const Product product = std::initializer_list<Product>{moe_product_b2, moe_product_b3, moe_product_b4,
                                                           moe_product_b5, moe_product_b6, moe_product_b8}.begin()[at];
    const Pack pack = std::initializer_list<Pack>{moe_pack_b2, moe_pack_b3, moe_pack_b4,
                                                  moe_pack_b5, moe_pack_b6, moe_pack_b8}.begin()[at];
    MoeParams p = {x.gate_words_dev, x.up_words_dev, x.gate_scales_dev, x.up_scales_dev,
                   x.gate_biases_dev, x.up_biases_dev, a.ids, a.x, h, (int)a.T, a.top_k, (int)x.E,
                   (int)x.inner, (int)x.K, x.group_size, a.dtype, nullptr};
    cudaError_t e;
    int variant = up_variant(&x, a.T, a.top_k);
    if (moe_packed(variant)) {
        e = pack(p, true, ws + w.x, a.stream);
        if (e != cudaSuccess) return e;
        p.packed = ws + w.x;
    }
    e = product(p, true, variant, a.stream);
    if (e != cudaSuccess) return e;
    p.w0 = p.w1 = x.down_words_dev;
    p.s0 = p.s1 = x.down_scales_dev;
    p.b0 = p.b1 = x.down_biases_dev;
    p.src = h;
    p.dst = parts;
    p.R = (int)x.K;
    p.K = (int)x.inner;
    p.packed = nullptr;
    variant = down_variant(&x, a.T, a.top_k);
    if (moe_packed(variant)) {
        e = pack(p, false, ws + w.hp, a.stream);
        if (e != cudaSuccess) return e;
        p.packed = ws + w.hp;
    }
    e = product(p, false, variant, a.stream);
    if (e != cudaSuccess) return e;
    const CombineParams c = {a.ids, a.weights, parts, a.out, (int)a.T, a.top_k, (int)x.E, (int)x.K,
                             a.dtype};
    const int64_t threads = a.T * (x.K / 4);
    return moe_launch(combine_kernel, dim3((unsigned)((threads + kThreads - 1) / kThreads)), kThreads,
                      0, 1, a.stream, c);
}

}  // namespace aq
