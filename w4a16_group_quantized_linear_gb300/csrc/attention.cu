// Attention of new tokens over a paged cache: which kernel serves which
// sequences, and a plain kernel for those of more rows than attention_step.cu
// takes: one warp per (token, query head), the head's elements spread over its lanes.
#include "attention.cuh"

namespace w4a16 {
namespace {

constexpr int kWarps = 4;

template <class E, int D>
__global__ void __launch_bounds__(kWarps * 32) attention_kernel(const __grid_constant__ AttentionArgs a, int min_rows) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (blockIdx.x == 0) check_offsets(a.c);
    constexpr int N = D / 64;  // element pairs per lane
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t t = row / a.heads;
    const int h = (int)(row % a.heads);
    if (t >= a.c.T) return;
    int first, count;
    const int b = sequence_of(a.c, t, first, count);
    if (b < 0) return;
    if (count * (a.heads / a.c.kv_heads) < min_rows) return;
    if (count > a.max_q_len) {
        raise_device_error(a.c.err, W4A16_ERR_BAD_OFFSETS);
        return;
    }
    const int length = cache_length(a.c, b);
    const int place = length - count + (int)(t - first);
    const int end = a.causal ? min(length, place + 1) : length;
    const int begin = a.window > 0 ? max(0, place - a.window + 1) : 0;
    const int g = h / (a.heads / a.c.kv_heads);

    float2 q[N], o[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        q[n] = E::unpack(*reinterpret_cast<const uint32_t*>(a.q + t * a.q_row_stride + h * a.q_head_stride +
                                                            2 * (n * 32 + lane)));
        o[n] = make_float2(0.0f, 0.0f);
    }
    float m = -INFINITY, l = 0.0f;
    for (int p = begin; p < end; ++p) {
        const int64_t page = page_of(a.c, b, p);
        if (page < 0) continue;
        const int64_t at = page * a.c.page_stride + (p % a.c.page_size) * a.c.slot_stride + g * a.c.head_stride;
        float s = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float2 k = E::unpack(*reinterpret_cast<const uint32_t*>(a.c.k + at + 2 * (n * 32 + lane)));
            s += q[n].x * k.x + q[n].y * k.y;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale_log2;
        const float top = fmaxf(m, s);
        const float keep = m == -INFINITY ? 0.0f : exp2f(m - top), w = exp2f(s - top);
        m = top;
        l = l * keep + w;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float2 v = E::unpack(*reinterpret_cast<const uint32_t*>(a.c.v + at + 2 * (n * 32 + lane)));
            o[n].x = o[n].x * keep + w * v.x;
            o[n].y = o[n].y * keep + w * v.y;
        }
    }
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n)
        *reinterpret_cast<uint32_t*>(a.out + (t * a.heads + h) * D + 2 * (n * 32 + lane)) =
            E::pack(o[n].x * inv, o[n].y * inv);
    if (a.lse && lane == 0) a.lse[t * a.heads + h] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

size_t attention_workspace_bytes(const DeviceInfo& dev, int64_t T, int batch, int heads, int kv_heads, int head_dim,
                                 int64_t max_q_len) {
    return attention_step_workspace_bytes(dev, head_dim);
}

w4a16_status attention_launch(const DeviceInfo& dev, int dtype, const AttentionArgs& a, void* workspace,
                              size_t workspace_bytes, cudaStream_t st) {
    const int64_t ratio = a.heads / a.c.kv_heads, most = a.max_q_len * ratio;
    if (workspace_bytes < attention_step_workspace_bytes(dev, a.c.head_dim) || !workspace) return W4A16_ERR_WORKSPACE;
    // where every sequence has the same number of new tokens, one kernel takes them all
    const bool alike = a.c.T == a.c.batch * a.max_q_len;
    const bool step = most <= kStepRows || (ratio <= kStepRows && !alike);
    const bool rest = most > kStepRows;
    if (step) {
        const w4a16_status s =
            attention_step_launch(dev, dtype, a, (int)(most < kStepRows ? most : kStepRows), workspace, st);
        if (s != W4A16_OK || !rest) return s;
    }
    const int64_t blocks = (a.c.T * a.heads + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return W4A16_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks);
    const bool f16 = dtype == W4A16_DTYPE_F16;
    const int min_rows = step ? kStepRows + 1 : 0;
    if (a.c.head_dim == 64)
        return launch_overlapped("paged_attention", f16 ? attention_kernel<Fp16, 64> : attention_kernel<Bf16, 64>, grid,
                                 kWarps * 32, 0, st, a, min_rows);
    return launch_overlapped("paged_attention", f16 ? attention_kernel<Fp16, 128> : attention_kernel<Bf16, 128>, grid,
                             kWarps * 32, 0, st, a, min_rows);
}

}  // namespace w4a16
