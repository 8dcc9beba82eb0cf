// The batch attention's own-keys kernel for 8-bit caches, head dimensions 64 and 128.
#include "aq_batch_host.cuh"

namespace aq {

cudaError_t batch_own8a(int64_t D, int group, const BatchRun &r) {
    if (D == 64 && group == 32) return own_run<8, 64, 32>(r);
    if (D == 64 && group == 64) return own_run<8, 64, 64>(r);
    if (D == 128 && group == 32) return own_run<8, 128, 32>(r);
    if (D == 128 && group == 64) return own_run<8, 128, 64>(r);
    if (D == 128 && group == 128) return own_run<8, 128, 128>(r);
    return cudaErrorInvalidValue;
}

}  // namespace aq
