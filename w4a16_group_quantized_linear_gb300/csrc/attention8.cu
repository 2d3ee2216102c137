// Attention of new tokens over a paged 8-bit cache: the kernels of the plan.
#include "attention_plan.cuh"
#include "cache8.cuh"

namespace w4a16 {

w4a16_status attention8_launch(const DeviceInfo& dev, int dtype, int format, const AttentionArgs& a,
                               const ScaleArgs& s, void* workspace, size_t workspace_bytes, cudaStream_t st) {
    if (!workspace || workspace_bytes < attention_workspace_bytes(dev, a.c.T, a.c.batch, a.heads, a.c.kv_heads,
                                                                  a.c.head_dim, a.max_q_len))
        return W4A16_ERR_WORKSPACE;
    const Plan p = plan_for(a.c.T, a.c.batch, a.heads, a.c.kv_heads, a.max_q_len, kStepRows8);
    if (p.step) {
        const w4a16_status e = attention8_step_launch(dev, dtype, format, a, s, p.step_rows, workspace, st);
        if (e != W4A16_OK || !p.tile) return e;
    }
    return attention8_tile_launch(dev, dtype, format, a, s, p.step ? kStepRows8 + 1 : 1,
                                  static_cast<unsigned char*>(workspace) +
                                      align_up(attention_step_workspace_bytes(dev, 128)), st);
}

}  // namespace w4a16
