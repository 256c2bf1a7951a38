// Token draw from bf16 logits (sample_kernel.cuh).
#include "sample_kernel.cuh"

namespace devscan {

cudaError_t launch_sample_bf16(const SampleCall &call, const Workspace &ws, cudaStream_t s)
{
    return launch_typed<__nv_bfloat16>(call, ws, s);
}

}  // namespace devscan
