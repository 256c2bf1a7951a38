// Token draw from f32 logits (sample_kernel.cuh).
#include "sample_kernel.cuh"

namespace devscan {

cudaError_t launch_sample_f32(const SampleCall &call, const Workspace &ws, cudaStream_t s)
{
    return launch_typed<float>(call, ws, s);
}

}  // namespace devscan
