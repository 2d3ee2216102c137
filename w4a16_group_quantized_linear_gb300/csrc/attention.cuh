// Declarations shared by the attention operators: 16-bit element types, the
// paged cache as the kernels see it, and the launch helper.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.cuh"
#include "sm100_ptx.cuh"

namespace w4a16 {

// ------------------------------------------------------- 16-bit elements --

struct Fp16 {
    static constexpr int kDtype = W4A16_DTYPE_F16;
    __device__ static __forceinline__ float2 unpack(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2*>(&v));
    }
    __device__ static __forceinline__ uint32_t pack(float lo, float hi) {  // round to nearest even
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

struct Bf16 {
    static constexpr int kDtype = W4A16_DTYPE_BF16;
    __device__ static __forceinline__ float2 unpack(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
    __device__ static __forceinline__ uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

// ---------------------------------------------------------------- cache --

// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery's method
// for a divisor known before the loop; here the host knows it).
struct FastDiv {
    uint32_t d, mul, shift;
    __device__ __forceinline__ int quotient(int n) const {
        return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift);
    }
    __device__ __forceinline__ int remainder(int n) const { return n - quotient(n) * (int)d; }
};

inline FastDiv fast_div(int divisor) {
    FastDiv f{(uint32_t)divisor, 0, 0};
    while ((1ull << f.shift) < f.d) ++f.shift;
    f.mul = (uint32_t)((1ull << 32) * ((1ull << f.shift) - f.d) / f.d + 1);
    return f;
}

// The paged cache and the batch that is appended to it or attends over it.
// Strides are in elements; element (page, slot, head, d) of either cache sits
// at page * page_stride + slot * slot_stride + head * head_stride + d.
struct CacheArgs {
    uint16_t* k;
    uint16_t* v;
    int64_t pages, page_stride, slot_stride, head_stride;
    const int32_t* table;   // [batch, table_stride], max_pages entries used of each row
    int64_t table_stride;
    int32_t page_size, max_pages;
    FastDiv by_page;  // the page size
    const int32_t* q_offsets;  // [batch + 1]
    const int32_t* kv_lens;    // [batch]
    int32_t batch, kv_heads, head_dim;
    int64_t T;
    unsigned int* err;
};

// Cached tokens of a sequence (n of kv_lens), held to what its row of the page table can name.
__device__ __forceinline__ int cache_length(const CacheArgs& c, int n) {
    const int64_t most = (int64_t)c.max_pages * c.page_size;
    if (n < 0 || n > most) {
        raise_device_error(c.err, W4A16_ERR_BAD_CACHE);
        return n < 0 ? 0 : (int)most;
    }
    return n;
}

// The sequence of token t, or -1 (reported) where the offsets are not a partition of the tokens.
__device__ __forceinline__ int sequence_of(const CacheArgs& c, int64_t t, int& first, int& count) {
    int b;
    if (c.T == c.batch) {
        b = (int)t;  // one token each, unless a sequence is empty
        first = __ldg(c.q_offsets + b);
        count = __ldg(c.q_offsets + b + 1) - first;
        if (first == t && count == 1) return b;
    }
    // the last b with q_offsets[b] <= t, for the warp's first token: 32 candidates at a time
    const int lane = threadIdx.x & 31;
    const unsigned active = __activemask();
    const int64_t t0 = __shfl_sync(active, t, __ffs(active) - 1);
    int lo = 0, width = c.batch;  // it is in [lo, lo + width)
    while (width > 1) {
        const int step = (width + 31) / 32;
        const int at = lo + lane * step;
        const bool le = at < lo + width && __ldg(c.q_offsets + at) <= t0;
        const unsigned hits = __ballot_sync(active, le);
        const int last = hits ? 31 - __clz(hits) : 0;
        width = min(step, width - last * step);
        lo += last * step;
    }
    b = lo;
    while (b + 1 < c.batch && __ldg(c.q_offsets + b + 1) <= t) ++b;  // this thread's, a token or two on
    first = __ldg(c.q_offsets + b);
    const int next = __ldg(c.q_offsets + b + 1);
    count = next - first;
    if (first < 0 || t < first || t >= next) {
        raise_device_error(c.err, W4A16_ERR_BAD_OFFSETS);
        return -1;
    }
    return b;
}

// Reports offsets that are not 0 = o[0] <= ... <= o[batch] = T; called by all
// threads of one block of a launch.
__device__ __forceinline__ void check_offsets(const CacheArgs& c) {
    bool ok = true;
    for (int b = threadIdx.x; b < c.batch; b += blockDim.x) {
        const int o = __ldg(c.q_offsets + b), next = __ldg(c.q_offsets + b + 1);
        ok = ok && o <= next && (b > 0 || o == 0) && (b < c.batch - 1 || next == c.T);
    }
    if (!ok) raise_device_error(c.err, W4A16_ERR_BAD_OFFSETS);
}

// Page that holds place p of sequence b, or -1 (reported) for an entry outside the cache.
__device__ __forceinline__ int64_t page_of(const CacheArgs& c, int b, int p) {
    const int32_t page = __ldg(c.table + b * c.table_stride + c.by_page.quotient(p));
    if (page < 0 || page >= c.pages) {
        raise_device_error(c.err, W4A16_ERR_BAD_CACHE);
        return -1;
    }
    return page;
}

// ------------------------------------------------------------------ host --

// Launches a kernel that may start while the one before it on the stream is
// still running (it waits for that one's results itself, before it reads).
template <typename... KArgs, typename... Args>
w4a16_status launch_overlapped(const char* what, void (*kernel)(KArgs...), dim3 grid, unsigned block, size_t smem,
                               cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attrs[1];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...), what);
}

w4a16_status rope_launch(const DeviceInfo& dev, int dtype, const uint16_t* x, int64_t x_row_stride,
                         int64_t x_head_stride, uint16_t* out, int64_t out_row_stride, int64_t out_head_stride,
                         int64_t T, int heads, int head_dim, const w4a16_rotary* rotary, cudaStream_t st);
w4a16_status append_launch(const DeviceInfo& dev, int dtype, const CacheArgs& c, const uint16_t* q,
                           int64_t q_row_stride, int64_t q_head_stride, int heads, uint16_t* q_out,
                           const uint16_t* k, int64_t k_row_stride, int64_t k_head_stride, const uint16_t* v,
                           int64_t v_row_stride, int64_t v_head_stride, const w4a16_rotary* rotary,
                           cudaStream_t st);

struct AttentionArgs {
    CacheArgs c;
    const uint16_t* q;
    int64_t q_row_stride, q_head_stride;
    uint16_t* out;  // [T, heads, head_dim]
    float* lse;     // [T, heads] or nullptr
    int32_t heads, ratio;   // ratio: query heads per cached head
    FastDiv by_ratio;       // T * ratio fits 31 bits
    int32_t causal, window;  // window 0: no lower limit
    float scale_log2;        // softmax scale times log2(e)
    int64_t max_q_len;
};

// The first place that a row at `place` sees. A row of a sequence that is shorter than its new tokens has a
// negative place, and the window may be anything up to 2^31 - 1: nothing here passes 32 bits.
__device__ __forceinline__ int first_seen(const AttentionArgs& a, int place) {
    const int back = a.window - 1;
    return a.window > 0 ? max(place, back) - back : 0;
}

// 2^x of the special-function unit (2 ulp), results below the normal range to zero.
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x 2^d for d <= 0, for a large x that is not to be lost with a 2^d below the normal range.
__device__ __forceinline__ float times_exp2(float x, float d) {
    float f = fast_exp2(d);
    if (d < -100.0f) {
        x *= 7.8886090522101181e-31f;  // 2^-100
        f = fast_exp2(d + 100.0f);
    }
    return x * f;
}

// Equal runs of a work list over the thread blocks: the first `more` take base + 1 units.
struct Shares {
    int64_t base;
    int more;
    __device__ __forceinline__ int64_t start(int c) const { return c * base + min(c, more); }
    // the thread block whose run holds the unit, looked for from block c on (a few steps: an
    // item is seldom cut into many parts, and a division here costs more)
    __device__ __forceinline__ int owner(int64_t unit, int c) const {
        while (start(c) > unit) --c;
        while (start(c + 1) <= unit) ++c;
        return c;
    }
};

constexpr size_t align_up(size_t n) { return (n + 255) & ~(size_t)255; }

// Sequences of up to kStepRows rows per cached head (attention_step.cu). max_rows
// is at least the rows of each of these sequences.
constexpr int kStepRows = 16;
w4a16_status attention_step_launch(const DeviceInfo& dev, int dtype, const AttentionArgs& a, int max_rows,
                                   void* workspace, cudaStream_t st);
size_t attention_step_workspace_bytes(const DeviceInfo& dev, int head_dim);

// Sequences of at least min_rows rows per cached head (attention_tile.cu).
w4a16_status attention_tile_launch(const DeviceInfo& dev, int dtype, const AttentionArgs& a, int min_rows,
                                   void* workspace, cudaStream_t st);
size_t attention_tile_workspace_bytes(const DeviceInfo& dev, int head_dim);

w4a16_status attention_launch(const DeviceInfo& dev, int dtype, const AttentionArgs& a, void* workspace,
                              size_t workspace_bytes, cudaStream_t st);
size_t attention_workspace_bytes(const DeviceInfo& dev, int64_t T, int batch, int heads, int kv_heads, int head_dim,
                                 int64_t max_q_len);

}  // namespace w4a16
