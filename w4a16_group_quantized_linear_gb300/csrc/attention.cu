// Attention of new tokens over a paged 16-bit cache: the kernels of its plan.
#include "attention_plan.cuh"

namespace w4a16 {

size_t attention_workspace_bytes(const DeviceInfo& dev, int64_t T, int batch, int heads, int kv_heads, int head_dim,
                                 int64_t max_q_len) {
    const Plan p = plan_for(T, batch, heads, kv_heads, max_q_len, kStepRows);
    return align_up(attention_step_workspace_bytes(dev, 128)) +
           (p.tile ? attention_tile_workspace_bytes(dev, head_dim) : 0);
}

w4a16_status attention_launch(const DeviceInfo& dev, int dtype, const AttentionArgs& a, void* workspace,
                              size_t workspace_bytes, cudaStream_t st) {
    if (!workspace || workspace_bytes < attention_workspace_bytes(dev, a.c.T, a.c.batch, a.heads, a.c.kv_heads,
                                                                  a.c.head_dim, a.max_q_len))
        return W4A16_ERR_WORKSPACE;
    const Plan p = plan_for(a.c.T, a.c.batch, a.heads, a.c.kv_heads, a.max_q_len, kStepRows);
    if (p.step) {
        const w4a16_status s = attention_step_launch(dev, dtype, a, p.step_rows, workspace, st);
        if (s != W4A16_OK || !p.tile) return s;
    }
    return attention_tile_launch(dev, dtype, a, p.step ? kStepRows + 1 : 1,
                                 static_cast<unsigned char*>(workspace) +
                                     align_up(attention_step_workspace_bytes(dev, 128)), st);
}

}  // namespace w4a16
