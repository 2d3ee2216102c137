// Attention for many rows over a 16-bit cache: the kernel is attention_tile.cuh's.
#include "attention_tile.cuh"

namespace w4a16 {

size_t attention_tile_workspace_bytes(const DeviceInfo& dev, int head_dim) {
    const size_t n = (size_t)dev.sms;
    return align_up(2 * n * sizeof(int)) + align_up(2 * n * kTile * sizeof(float2)) +
           2 * n * kTile * head_dim * sizeof(float);
}

w4a16_status attention_tile_launch(const DeviceInfo& dev, int dtype, const AttentionArgs& a, int min_rows,
                                   void* workspace, cudaStream_t st) {
    const TileArgs x = tile_args(dev, a, ScaleArgs{}, min_rows, workspace);
    const bool f16 = dtype == W4A16_DTYPE_F16;
    return f16 ? launch_dim<Fp16, Held16>(dev, x, st) : launch_dim<Bf16, Held16>(dev, x, st);
}

#ifdef W4A16_TEST_HOOKS
cudaError_t attention_set_test_hooks(const TestHooks& h) { return cudaMemcpyToSymbol(g_hooks, &h, sizeof(h)); }
cudaError_t attention_get_test_counters(TestCounters* c) { return cudaMemcpyFromSymbol(c, g_counters, sizeof(*c)); }
#endif

}  // namespace w4a16
