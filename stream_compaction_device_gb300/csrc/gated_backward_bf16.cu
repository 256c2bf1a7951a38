// The gated recurrence's gradient on bf16 values (a translation unit per type and direction,
// compiled in parallel).
#include "gated_scan.cuh"

namespace devscan {

cudaError_t launch_gated_backward_bf16(const GatedBackwardCall &call, bool wide, int sms, cudaStream_t s)
{
    return wide ? gated::backward_any<__nv_bfloat16, float>(call, sms, s) : gated::backward_any<__nv_bfloat16, __nv_bfloat16>(call, sms, s);
}

}  // namespace devscan
