// Token draw from f16 logits (sample_kernel.cuh).
#include "sample_kernel.cuh"

namespace devscan {

cudaError_t launch_sample_f16(const SampleCall &call, const Workspace &ws, cudaStream_t s)
{
    return launch_typed<__half>(call, ws, s);
}

}  // namespace devscan
