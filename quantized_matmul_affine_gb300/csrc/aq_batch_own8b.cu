// The batch attention's own-keys kernel for 8-bit caches, head dimensions 256 and 512.
#include "aq_batch_host.cuh"

namespace aq {

cudaError_t batch_own8b(int64_t D, int group, const BatchRun &r) {
    if (D == 256 && group == 32) return own_run<8, 256, 32>(r);
    if (D == 256 && group == 64) return own_run<8, 256, 64>(r);
    if (D == 256 && group == 128) return own_run<8, 256, 128>(r);
    if (D == 512 && group == 32) return own_run<8, 512, 32>(r);
    if (D == 512 && group == 64) return own_run<8, 512, 64>(r);
    if (D == 512 && group == 128) return own_run<8, 512, 128>(r);
    return cudaErrorInvalidValue;
}

}  // namespace aq
