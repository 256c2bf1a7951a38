// The gated recurrence on f32 values (a translation unit per type and direction,
// compiled in parallel).
#include "gated_scan.cuh"

namespace devscan {

cudaError_t launch_gated_scan_f32(const GatedScanCall &call, bool , int sms, cudaStream_t s)
{
    return gated::forward_any<float, float>(call, sms, s);
}

}  // namespace devscan
