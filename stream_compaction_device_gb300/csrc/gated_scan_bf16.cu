// The gated recurrence on bf16 values (a translation unit per type and direction,
// compiled in parallel).
#include "gated_scan.cuh"

namespace devscan {

cudaError_t launch_gated_scan_bf16(const GatedScanCall &call, bool wide, int sms, cudaStream_t s)
{
    return wide ? gated::forward_any<__nv_bfloat16, float>(call, sms, s) : gated::forward_any<__nv_bfloat16, __nv_bfloat16>(call, sms, s);
}

}  // namespace devscan
