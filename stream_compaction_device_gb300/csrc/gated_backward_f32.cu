// The gated recurrence's gradient on f32 values (a translation unit per type and direction,
// compiled in parallel).
#include "gated_scan.cuh"

namespace devscan {

cudaError_t launch_gated_backward_f32(const GatedBackwardCall &call, bool , int sms, cudaStream_t s)
{
    return gated::backward_any<float, float>(call, sms, s);
}

}  // namespace devscan
