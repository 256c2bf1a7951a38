// The gated recurrence on f16 values (a translation unit per type and direction,
// compiled in parallel).
#include "gated_scan.cuh"

namespace devscan {

cudaError_t launch_gated_scan_f16(const GatedScanCall &call, bool wide, int sms, cudaStream_t s)
{
    return wide ? gated::forward_any<__half, float>(call, sms, s) : gated::forward_any<__half, __half>(call, sms, s);
}

}  // namespace devscan
