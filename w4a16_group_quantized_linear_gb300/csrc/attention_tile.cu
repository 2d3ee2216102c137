// Attention for many rows over a 16-bit cache: the kernel is attention_tile.cuh's.
#include <cudaTypedefs.h>

#include <mutex>

#include "attention_tile.cuh"

namespace w4a16 {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// [pages][heads][slots][elements] of k or v, boxes of 64 elements of `box` slots
w4a16_status make_map(const CacheArgs& c, const uint16_t* base, bool f16, int box, CUtensorMap* map) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc) return cuda_status(cudaErrorNotSupported, "paged_attention: cuTensorMapEncodeTiled entry point");
    cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.kv_heads,
                          (cuuint64_t)c.pages};
    cuuint64_t strides[3] = {(cuuint64_t)c.slot_stride * 2, (cuuint64_t)c.head_stride * 2,
                             (cuuint64_t)c.page_stride * 2};
    cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    if (enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<uint16_t*>(base), dims, strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cuda_status(cudaErrorInvalidValue, "paged_attention: cuTensorMapEncodeTiled");
    return W4A16_OK;
}

template <class E, int D, bool PAIRED>
w4a16_status launch(const DeviceInfo& dev, const TileArgs& x, cudaStream_t st) {
    CUtensorMap mk, mv;
    const bool f16 = E::kDtype == W4A16_DTYPE_F16;
    w4a16_status s = make_map(x.a.c, x.a.c.k, f16, x.box, &mk);
    if (s == W4A16_OK) s = make_map(x.a.c, x.a.c.v, f16, x.box, &mv);
    if (s != W4A16_OK) return s;
    return launch_with_maps<E, Held16, D, PAIRED>(dev, mk, mv, x, st);
}

template <class E, int D>
w4a16_status launch_rows(const DeviceInfo& dev, const TileArgs& x, cudaStream_t st) {
    // Sequences that all fit half a tile (drafts being verified, short chunks)
    // share out their blocks between the halves: 5 tokens x 5 heads over 2000 to
    // 9000 places, 16 sequences, 87 us against 103 with one half idle (and the
    // maximum that lags). For tiles of both halves the issuing loop that
    // knows of no pairs is the faster one (2048 tokens over 30048 places 807
    // against 868 us when both were built with that maximum).
    return x.a.max_q_len * x.a.ratio <= kHalf ? launch<E, D, true>(dev, x, st) : launch<E, D, false>(dev, x, st);
}

}  // namespace

size_t attention_tile_workspace_bytes(const DeviceInfo& dev, int head_dim) {
    const size_t n = (size_t)dev.sms;
    return align_up(2 * n * sizeof(int)) + align_up(2 * n * kTile * sizeof(float2)) +
           2 * n * kTile * head_dim * sizeof(float);
}

w4a16_status attention_tile_launch(const DeviceInfo& dev, int dtype, const AttentionArgs& a, int min_rows,
                                   void* workspace, cudaStream_t st) {
    const TileArgs x = tile_args(dev, a, ScaleArgs{}, min_rows, workspace);
    const bool f16 = dtype == W4A16_DTYPE_F16;
    if (a.c.head_dim == 128) return f16 ? launch_rows<Fp16, 128>(dev, x, st) : launch_rows<Bf16, 128>(dev, x, st);
    return f16 ? launch_rows<Fp16, 64>(dev, x, st) : launch_rows<Bf16, 64>(dev, x, st);
}

#ifdef W4A16_TEST_HOOKS
cudaError_t attention_set_test_hooks(const TestHooks& h) { return cudaMemcpyToSymbol(g_hooks, &h, sizeof(h)); }
cudaError_t attention_get_test_counters(TestCounters* c) { return cudaMemcpyFromSymbol(c, g_counters, sizeof(*c)); }
#endif

}  // namespace w4a16
