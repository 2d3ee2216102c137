// Attention of new tokens over a paged cache of 8-bit rows: one warp per row
// (query head of a new token), the places in order, with the running maximum of the softmax.
#include "attention_plan.cuh"
#include "cache8.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 128;

struct Args8 {
    AttentionArgs a;
    ScaleArgs s;
    int min_rows;  // sequences with fewer rows per cached head are attention8_step.cu's
};

template <class E, class H, int D>
__global__ void __launch_bounds__(kThreads) row_kernel(const __grid_constant__ Args8 x) {
    const AttentionArgs& a = x.a;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (blockIdx.x == 0) check_offsets(a.c);
    constexpr int kPer = D / 32;  // elements a lane
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = row / a.heads;
    const int h = (int)(row % a.heads), g = h / a.ratio;
    if (t >= a.c.T) return;
    int first, count;
    const int b = sequence_of(a.c, t, first, count);
    if (b < 0) return;
    if (count > a.max_q_len) {
        raise_device_error(a.c.err, W4A16_ERR_BAD_OFFSETS);
        return;
    }
    if (count * a.ratio < x.min_rows) return;
    const int length = cache_length(a.c, __ldg(a.c.kv_lens + b));
    const int place = length - count + (int)(t - first);
    const int high = a.causal ? min(length, place + 1) : length;
    float q[kPer], o[kPer];
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
        const float2 v = E::unpack(*reinterpret_cast<const uint32_t*>(a.q + t * a.q_row_stride + h * a.q_head_stride +
                                                                      lane * kPer + 2 * i));
        q[2 * i] = v.x;
        q[2 * i + 1] = v.y;
        o[2 * i] = o[2 * i + 1] = 0.0f;
    }
    auto load = [&](const uint16_t* base, int64_t off, float (&v)[kPer]) {
        const uint8_t* src = reinterpret_cast<const uint8_t*>(base) + off + lane * kPer;
        float w[4];
        H::decode4(kPer == 4 ? *reinterpret_cast<const uint32_t*>(src) : *reinterpret_cast<const uint16_t*>(src), w);
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = w[i];
    };
    float m = -INFINITY, l = 0.0f;
    for (int p = first_seen(a, place); p < high; ++p) {
        const int64_t page = page_of(a.c, b, p);
        if (page < 0) continue;
        const int in_page = a.c.by_page.remainder(p);
        const int64_t off = page * a.c.page_stride + in_page * a.c.slot_stride + g * a.c.head_stride;
        const int64_t scale = page * x.s.page_stride + g * x.s.head_stride + in_page;
        float k[kPer], v[kPer], s = 0.0f;
        load(a.c.k, off, k);
        load(a.c.v, off, v);
#pragma unroll
        for (int i = 0; i < kPer; ++i) s += q[i] * k[i];
        for (int d = 1; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale_log2 * x.s.k[scale];
        const float top = fmaxf(m, s), keep = m == -INFINITY ? 0.0f : fast_exp2(m - top);
        const float w = fast_exp2(s - (top == -INFINITY ? 0.0f : top)), wv = w * x.s.v[scale];
        l = l * keep + w;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = o[i] * keep + wv * v[i];
        m = top;
    }
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i)
        *reinterpret_cast<uint32_t*>(a.out + (t * a.heads + h) * D + lane * kPer + 2 * i) =
            E::pack(o[2 * i] * inv, o[2 * i + 1] * inv);
    if (a.lse && lane == 0) a.lse[t * a.heads + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <class E, class H>
w4a16_status launch(const Args8& x, cudaStream_t st) {
    const int64_t blocks = (x.a.c.T * x.a.heads + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffffLL) return W4A16_ERR_UNSUPPORTED;
    return launch_overlapped("paged_attention", x.a.c.head_dim == 128 ? row_kernel<E, H, 128> : row_kernel<E, H, 64>,
                             dim3((unsigned)blocks), kThreads, 0, st, x);
}

}  // namespace

w4a16_status attention8_launch(const DeviceInfo& dev, int dtype, int format, const AttentionArgs& a,
                               const ScaleArgs& s, void* workspace, size_t workspace_bytes, cudaStream_t st) {
    if (!workspace || workspace_bytes < attention_workspace_bytes(dev, a.c.T, a.c.batch, a.heads, a.c.kv_heads,
                                                                  a.c.head_dim, a.max_q_len))
        return W4A16_ERR_WORKSPACE;
    const Plan p = plan_for(a.c.T, a.c.batch, a.heads, a.c.kv_heads, a.max_q_len);
    if (p.step) {
        const w4a16_status e = attention8_step_launch(dev, dtype, format, a, s, p.step_rows, workspace, st);
        if (e != W4A16_OK || !p.tile) return e;
    }
    const Args8 x{a, s, p.step ? kStepRows + 1 : 1};
    const bool f16 = dtype == W4A16_DTYPE_F16;
    if (format == W4A16_CACHE_INT8) return f16 ? launch<Fp16, HeldInt8>(x, st) : launch<Bf16, HeldInt8>(x, st);
    return f16 ? launch<Fp16, HeldE4m3>(x, st) : launch<Bf16, HeldE4m3>(x, st);
}

}  // namespace w4a16
