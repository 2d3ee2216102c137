// Attention of new tokens over a paged cache: which kernel serves which sequences.
//
// A sequence's work is a number of rows per cached head: its new tokens times
// the query heads that share the head. With few rows the cache's bytes are all
// that counts and attention_step.cu takes them; past 16 the 8-row products
// of that kernel are what it waits for (with a variant for 32 rows, 25 rows of
// 16 sequences took 94 us, where the tiles take 87, and 32 of 64 sequences 132
// against 130), and attention_tile.cu takes 256 rows to a tile on the tensor
// cores. The lengths are on the device, so where a batch may hold both kinds
// both kernels are launched, and each passes over the other's.
#include "attention.cuh"

namespace w4a16 {
namespace {

struct Plan {
    bool step, tile;
    int step_rows;  // most rows of a sequence of the step kernel
};

Plan plan_for(int64_t T, int64_t batch, int heads, int kv_heads, int64_t max_q_len) {
    const int64_t ratio = heads / kv_heads, most = (max_q_len < T ? max_q_len : T) * ratio;
    Plan p;
    p.tile = most > kStepRows;
    // every sequence has max_q_len new tokens, as one alone has: no second kind
    const bool alike = T == batch * max_q_len || batch == 1;
    p.step = !p.tile || (ratio <= kStepRows && !alike);
    p.step_rows = (int)(most < kStepRows ? most : kStepRows);
    return p;
}

}  // namespace

size_t attention_workspace_bytes(const DeviceInfo& dev, int64_t T, int batch, int heads, int kv_heads, int head_dim,
                                 int64_t max_q_len) {
    const Plan p = plan_for(T, batch, heads, kv_heads, max_q_len);
    return align_up(attention_step_workspace_bytes(dev, 128)) +
           (p.tile ? attention_tile_workspace_bytes(dev, head_dim) : 0);
}

w4a16_status attention_launch(const DeviceInfo& dev, int dtype, const AttentionArgs& a, void* workspace,
                              size_t workspace_bytes, cudaStream_t st) {
    if (!workspace || workspace_bytes < attention_workspace_bytes(dev, a.c.T, a.c.batch, a.heads, a.c.kv_heads,
                                                                  a.c.head_dim, a.max_q_len))
        return W4A16_ERR_WORKSPACE;
    const Plan p = plan_for(a.c.T, a.c.batch, a.heads, a.c.kv_heads, a.max_q_len);
    if (p.step) {
        const w4a16_status s = attention_step_launch(dev, dtype, a, p.step_rows, workspace, st);
        if (s != W4A16_OK || !p.tile) return s;
    }
    return attention_tile_launch(dev, dtype, a, p.step ? kStepRows + 1 : 1,
                                 static_cast<unsigned char*>(workspace) +
                                     align_up(attention_step_workspace_bytes(dev, 128)), st);
}

}  // namespace w4a16
