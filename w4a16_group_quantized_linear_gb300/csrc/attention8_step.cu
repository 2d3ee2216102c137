// Attention for few rows over an 8-bit cache: the kernel is attention_step.cuh's.
#include "attention_step.cuh"

namespace w4a16 {

w4a16_status attention8_step_launch(const DeviceInfo& dev, int dtype, int format, const AttentionArgs& a,
                                    const ScaleArgs& s, int max_rows, void* workspace, cudaStream_t st) {
    const bool f16 = dtype == W4A16_DTYPE_F16;
    if (format == W4A16_CACHE_INT8)
        return f16 ? launch_rows<Fp16, HeldInt8>(dev, a, s, max_rows, workspace, st)
                   : launch_rows<Bf16, HeldInt8>(dev, a, s, max_rows, workspace, st);
    return f16 ? launch_rows<Fp16, HeldE4m3>(dev, a, s, max_rows, workspace, st)
               : launch_rows<Bf16, HeldE4m3>(dev, a, s, max_rows, workspace, st);
}

}  // namespace w4a16
