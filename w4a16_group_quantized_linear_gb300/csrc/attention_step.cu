// Attention for few rows over a 16-bit cache: the kernel is attention_step.cuh's.
#include "attention_step.cuh"

namespace w4a16 {

size_t attention_step_workspace_bytes(const DeviceInfo& dev, int head_dim) {
    const size_t n = (size_t)step_blocks(dev);
    return align_up(n * sizeof(int)) + align_up(2 * n * kStepRows * sizeof(float2)) +
           2 * n * kStepRows * head_dim * sizeof(float);
}

w4a16_status attention_step_launch(const DeviceInfo& dev, int dtype, const AttentionArgs& a, int max_rows,
                                   void* workspace, cudaStream_t st) {
    return dtype == W4A16_DTYPE_F16 ? launch_rows<Fp16, Held16>(dev, a, ScaleArgs{}, max_rows, workspace, st)
                                    : launch_rows<Bf16, Held16>(dev, a, ScaleArgs{}, max_rows, workspace, st);
}

}  // namespace w4a16
