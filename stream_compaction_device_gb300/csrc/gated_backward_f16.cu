// The gated recurrence's gradient on f16 values (a translation unit per type and direction,
// compiled in parallel).
#include "gated_scan.cuh"

namespace devscan {

cudaError_t launch_gated_backward_f16(const GatedBackwardCall &call, bool wide, int sms, cudaStream_t s)
{
    return wide ? gated::backward_any<__half, float>(call, sms, s) : gated::backward_any<__half, __half>(call, sms, s);
}

}  // namespace devscan
