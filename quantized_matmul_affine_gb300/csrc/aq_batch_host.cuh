// Host side of the batch attention's own-keys kernel: launch geometry of one
// instantiation, included by the files that instantiate it.
#pragma once

#include "aq_batch_own.cuh"

#include <algorithm>
#include <mutex>

namespace aq {

struct BatchRun {
    BatchParams prm;
    int nb;              // blocks of 8 query rows a tile
    cudaStream_t stream;
    // planning only: CTAs the device holds at once, keys a tile
    int *resident, *unit_keys;
};

// (Without a name for the linker: what is kept once a kernel must not be
// shared with another copy of the library in the process.)
namespace {

template <int BITS, int D, int GROUP, int NB>
cudaError_t own_run_nb(const BatchRun &r) {
    using S = Own<BITS, D, GROUP, NB>;
    auto kern = own_kernel<BITS, D, GROUP, NB>;
    constexpr int smem = S::kSmem;
    static std::once_flag once;
    static cudaError_t attr = cudaSuccess;
    static int per_sm = 0;
    std::call_once(once, [&] {
        attr = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (attr == cudaSuccess)
            attr = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, S::kThreads, smem);
    });
    if (attr != cudaSuccess) return attr;
    if (r.resident) {
        *r.resident = per_sm * num_sms();
        *r.unit_keys = S::kKeys;
        return cudaSuccess;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(r.prm.own_warps / S::kWarps), 1, 1);
    cfg.blockDim = dim3(S::kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = r.stream;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = a;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, r.prm);
}

template <int BITS, int D, int GROUP>
cudaError_t own_run(const BatchRun &r) {
    if constexpr (D == 512)  // 128 accumulators a lane for one block of 8 rows
        return own_run_nb<BITS, D, GROUP, 1>(r);
    else
        return r.nb == 1 ? own_run_nb<BITS, D, GROUP, 1>(r) : own_run_nb<BITS, D, GROUP, 2>(r);
}

}  // namespace

cudaError_t batch_own4a(int64_t D, int group, const BatchRun &r);
cudaError_t batch_own4b(int64_t D, int group, const BatchRun &r);
cudaError_t batch_own8a(int64_t D, int group, const BatchRun &r);
cudaError_t batch_own8b(int64_t D, int group, const BatchRun &r);

}  // namespace aq
