// Attention for many rows over an 8-bit cache: the kernel is attention_tile.cuh's.
#include "attention_tile.cuh"

namespace w4a16 {

w4a16_status attention8_tile_launch(const DeviceInfo& dev, int dtype, int format, const AttentionArgs& a,
                                    const ScaleArgs& s, int min_rows, void* workspace, cudaStream_t st) {
    const TileArgs x = tile_args(dev, a, s, min_rows, workspace);
    const bool f16 = dtype == W4A16_DTYPE_F16;
    if (format == W4A16_CACHE_INT8)
        return f16 ? launch_dim<Fp16, HeldInt8>(dev, x, st) : launch_dim<Bf16, HeldInt8>(dev, x, st);
    return f16 ? launch_dim<Fp16, HeldE4m3>(dev, x, st) : launch_dim<Bf16, HeldE4m3>(dev, x, st);
}

#ifdef W4A16_TEST_HOOKS
cudaError_t attention8_set_test_hooks(const TestHooks& h) { return cudaMemcpyToSymbol(g_hooks, &h, sizeof(h)); }
cudaError_t attention8_get_test_counters(TestCounters* c) { return cudaMemcpyFromSymbol(c, g_counters, sizeof(*c)); }
#endif

}  // namespace w4a16
