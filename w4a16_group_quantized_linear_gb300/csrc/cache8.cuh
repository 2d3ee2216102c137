// The 8-bit paged cache as the kernels see it. A row x of head_dim elements is
// held as one byte an element and one fp32 scale:
//     s = max(max|x|, 2^-100) / most,   q = x / s rounded to nearest,   x ~ q s
// with q an integer in [-127, 127] (most = 127) or an e4m3 number (most = 448).
// The lower limit of the largest element keeps s and 1 / s normal numbers. A row
// that holds an infinity or a NaN has the scale NaN: it reads back as NaN.
#pragma once

#include "attention.cuh"

namespace w4a16 {

// Scale of slot `slot` of head g in a page: [page * page_stride + g * head_stride + slot].
struct ScaleArgs {
    float* k;
    float* v;
    int64_t page_stride, head_stride;
};

constexpr float kLeastTop = 7.8886090522101181e-31f;  // 2^-100

// 16-bit elements, for kernels that serve both kinds of cache.
struct Held16 {
    static constexpr int kFormat = 0;
};

struct HeldInt8 {
    static constexpr int kFormat = W4A16_CACHE_INT8;
    static constexpr float kMost = 127.0f;
    // x inv, |x inv| <= 127 but for rounding, to the nearest integers (ties to even): with
    // 1.5 * 2^23 added, an integer's two's complement is in the low bits of the sum
    __device__ static __forceinline__ uint32_t encode4(const float* x, float inv) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(__fadd_rn(__fmul_rn(x[i], inv), 12582912.0f));
        return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    __device__ static __forceinline__ void decode4(uint32_t v, float* x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(v >> (8 * i));
    }
    // Four of them as fp16 pairs, exactly: with its sign bit flipped a byte u is q + 128, and the low byte
    // of fp16's 1024 + u.
    __device__ static __forceinline__ uint32_t minus_1152(uint32_t v) {
        const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&v),
                                  __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ static __forceinline__ void to_fp16(uint32_t v, uint32_t& b01, uint32_t& b23) {
        v ^= 0x80808080u;
        b01 = minus_1152(__byte_perm(v, 0x64646464u, 0x4140));
        b23 = minus_1152(__byte_perm(v, 0x64646464u, 0x4342));
    }
    __device__ static __forceinline__ void to_fp16_apart(uint32_t v, uint32_t& b02, uint32_t& b13) {
        v ^= 0x80808080u;
        b02 = minus_1152(__byte_perm(v, 0x64646464u, 0x4240));
        b13 = minus_1152(__byte_perm(v, 0x64646464u, 0x4341));
    }
};

struct HeldE4m3 {
    static constexpr int kFormat = W4A16_CACHE_E4M3;
    static constexpr float kMost = 448.0f;
    __device__ static __forceinline__ uint32_t encode4(const float* x, float inv) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1] * inv), "f"(x[0] * inv));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3] * inv), "f"(x[2] * inv));
        return (uint32_t)lo | (uint32_t)hi << 16;
    }
    __device__ static __forceinline__ void to_fp16(uint32_t v, uint32_t& b01, uint32_t& b23) {
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(b01), "=r"(b23)
            : "r"(v));
    }
    __device__ static __forceinline__ void to_fp16_apart(uint32_t v, uint32_t& b02, uint32_t& b13) {
        to_fp16(__byte_perm(v, 0, 0x3120), b02, b13);
    }
    __device__ static __forceinline__ void decode4(uint32_t v, float* x) {
        uint32_t lo, hi;
        to_fp16(v, lo, hi);
        const float2 a = Fp16::unpack(lo), b = Fp16::unpack(hi);
        x[0] = a.x;
        x[1] = a.y;
        x[2] = b.x;
        x[3] = b.y;
    }
};

// The larger of two, NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Scale of a row and what its elements are multiplied by, from its largest |x| (NaN where one is). NaN
// where the row holds an infinity or a NaN.
template <class H>
__device__ __forceinline__ float scale_of(float top, float& inv) {
    const float held = fmaxf(top, kLeastTop);
    inv = __fdiv_rn(H::kMost, held);
    return top < INFINITY ? __fdiv_rn(held, H::kMost) : __uint_as_float(0x7FC00000u);
}

// ------------------------------------------------------------------ host --

w4a16_status rope_norm_launch(const DeviceInfo& dev, int dtype, const uint16_t* x, int64_t x_row_stride,
                              int64_t x_head_stride, uint16_t* out, int64_t out_row_stride, int64_t out_head_stride,
                              int64_t T, int heads, int head_dim, const float* weight, float eps,
                              const w4a16_rotary* rotary, cudaStream_t st);
// format: 0 (16 bits) or W4A16_CACHE_*
w4a16_status append_ex_launch(const DeviceInfo& dev, int dtype, int format, const CacheArgs& c, const ScaleArgs& s,
                              const uint16_t* q, int64_t q_row_stride, int64_t q_head_stride, int heads,
                              uint16_t* q_out, const uint16_t* k, int64_t k_row_stride, int64_t k_head_stride,
                              const uint16_t* v, int64_t v_row_stride, int64_t v_head_stride,
                              const w4a16_head_norms* norms, const w4a16_rotary* rotary, cudaStream_t st);
w4a16_status read_launch(const DeviceInfo& dev, int dtype, int format, const CacheArgs& c, const ScaleArgs& s,
                         uint16_t* k, uint16_t* v, cudaStream_t st);
// Sequences of up to kStepRows8 rows per cached head, in groups of kStepRows.
constexpr int kStepRows8 = 3 * kStepRows;
w4a16_status attention8_step_launch(const DeviceInfo& dev, int dtype, int format, const AttentionArgs& a,
                                    const ScaleArgs& s, int max_rows, void* workspace, cudaStream_t st);
w4a16_status attention8_tile_launch(const DeviceInfo& dev, int dtype, int format, const AttentionArgs& a,
                                    const ScaleArgs& s, int min_rows, void* workspace, cudaStream_t st);
w4a16_status attention8_launch(const DeviceInfo& dev, int dtype, int format, const AttentionArgs& a,
                               const ScaleArgs& s, void* workspace, size_t workspace_bytes, cudaStream_t st);

}  // namespace w4a16
