// Norms of the query and key heads with the position rotation in the same
// pass, the paged cache in 8 bits as it is appended to, and reading it back.
//
// A head x becomes  y = turn(x / sqrt(mean(x^2) + eps) * w)  and, in an 8-bit cache, a
// scale s and q = y / s (cache8.cuh), all in fp32 from the 16-bit input to the one rounding of
// the result. mean(x^2) and the largest |y| are over the head's 4 to 32 threads,
// of 16 elements each, by shuffles: their order is fixed.
//
// Like rope_cache.cu's, these kernels move bytes and do little else.
#include "cache8.cuh"
#include "rotary.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;

// The 16 elements of a thread, as 32-bit numbers.
template <class E>
__device__ __forceinline__ void unpack16(const uint4& u, const uint4& w, float (&x)[16]) {
    const uint32_t v[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 p = E::unpack(v[i]);
        x[2 * i] = p.x;
        x[2 * i + 1] = p.y;
    }
}

template <class E>
__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(E::pack(x[0], x[1]), E::pack(x[2], x[3]), E::pack(x[4], x[5]), E::pack(x[6], x[7]));
}

// x / sqrt(mean(x^2) + eps) * w over the `lanes` lanes of a head (w: the thread's two pieces).
__device__ __forceinline__ void normalise(float (&x)[16], int lanes, int head_dim, float eps, const float* w0,
                                          const float* w1) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += x[i] * x[i];
    for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float r = rsqrtf(sum / (float)head_dim + eps);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(w0) + i);
        const float4 b = __ldg(reinterpret_cast<const float4*>(w1) + i);
        x[4 * i] *= r * a.x;
        x[4 * i + 1] *= r * a.y;
        x[4 * i + 2] *= r * a.z;
        x[4 * i + 3] *= r * a.w;
        x[8 + 4 * i] *= r * b.x;
        x[8 + 4 * i + 1] *= r * b.y;
        x[8 + 4 * i + 2] *= r * b.z;
        x[8 + 4 * i + 3] *= r * b.w;
    }
}

// Turns the 8 pairs of the two pieces of 8 elements.
__device__ __forceinline__ void turn(float (&x)[16], bool interleaved, const float (&c)[8], const float (&s)[8]) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * c[i] - b * s[i];
            x[2 * i + 1] = b * c[i] + a * s[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = x[i], b = x[i + 8];
            x[i] = a * c[i] - b * s[i];
            x[i + 8] = b * c[i] + a * s[i];
        }
    }
}

// ------------------------------------------------------------------- rope --

struct NormArgs {
    const uint16_t* x;
    int64_t x_row_stride, x_head_stride;
    uint16_t* out;
    int64_t out_row_stride, out_head_stride;
    int64_t T;
    int32_t heads, head_dim, lanes;  // lanes: of a head, a power of two
    const float* weight;
    float eps;
    unsigned int* err;
    RotaryArgs r;
};

template <class E, int HPT>
__global__ void __launch_bounds__(kThreads) rope_norm_kernel(const __grid_constant__ NormArgs a) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int groups = (a.heads + HPT - 1) / HPT;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int chunk = (int)(i % a.lanes);
    const int group = (int)(i / a.lanes % groups);
    const int64_t t = i / a.lanes / groups;
    // the lanes of a head, and those past its end, stay together for the sums
    const bool mine = t < a.T && chunk < a.head_dim / 16;
    const Pieces p = pieces_of(a.r, mine ? chunk : 0);
    uint4 u[HPT], w[HPT];
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
        const int h = group + k * groups;
        u[k] = w[k] = make_uint4(0, 0, 0, 0);
        if (!mine || h >= a.heads) continue;
        const uint16_t* src = a.x + t * a.x_row_stride + h * a.x_head_stride;
        u[k] = *reinterpret_cast<const uint4*>(src + p.first);
        w[k] = *reinterpret_cast<const uint4*>(src + p.second);
    }
    float c[8], s[8];
    const bool rotate = mine && p.pair >= 0 && angles(a.r, a.T, t, 0, p.pair, a.err, c, s);
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
        const int h = group + k * groups;
        float x[16];
        unpack16<E>(u[k], w[k], x);
        normalise(x, a.lanes, a.head_dim, a.eps, a.weight + p.first, a.weight + p.second);
        if (rotate) turn(x, a.r.interleaved, c, s);
        if (!mine || h >= a.heads) continue;
        uint16_t* dst = a.out + t * a.out_row_stride + h * a.out_head_stride;
        *reinterpret_cast<uint4*>(dst + p.first) = pack8<E>(x);
        *reinterpret_cast<uint4*>(dst + p.second) = pack8<E>(x + 8);
    }
}

// ----------------------------------------------------------------- append --

struct AppendArgs {
    CacheArgs c;
    ScaleArgs s;
    const uint16_t *q, *k, *v;
    int64_t q_row_stride, q_head_stride, k_row_stride, k_head_stride, v_row_stride, v_head_stride;
    uint16_t* q_out;  // [T, heads, head_dim]
    int32_t heads;    // 0: no q
    const float *q_norm, *k_norm;  // nullptr: left as they are
    float eps;
    RotaryArgs r;
};

// The heads of a token in one row: queries, then keys, then values.
template <class E, class H, int HPT>
__global__ void __launch_bounds__(kThreads) append_ex_kernel(const __grid_constant__ AppendArgs a) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (blockIdx.x == 0) check_offsets(a.c);
    const int D = a.c.head_dim, G = a.c.kv_heads;
    const int chunks = D / 16;  // 4 or 8: a head's lanes are in one warp
    const int all = a.heads + 2 * G;
    const int groups = (all + HPT - 1) / HPT;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int chunk = (int)(i % chunks);
    const int group = (int)(i / chunks % groups);
    const bool real = i / chunks / groups < a.c.T;  // lanes without a token stay for the sums
    const int64_t t = real ? i / chunks / groups : a.c.T - 1;
    const Pieces p = pieces_of(a.r, chunk);
    uint4 u[HPT], w[HPT];
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
        const int h = group + k * groups;
        u[k] = w[k] = make_uint4(0, 0, 0, 0);
        if (!real || h >= all) continue;
        const uint16_t* src = h < a.heads ? a.q + t * a.q_row_stride + h * a.q_head_stride
                              : h < a.heads + G ? a.k + t * a.k_row_stride + (h - a.heads) * a.k_head_stride
                                                : a.v + t * a.v_row_stride + (h - a.heads - G) * a.v_head_stride;
        u[k] = *reinterpret_cast<const uint4*>(src + p.first);
        w[k] = *reinterpret_cast<const uint4*>(src + p.second);
    }
    int first, count;
    const int b = sequence_of(a.c, t, first, count);
    // place in the sequence; negative where the sequence is shorter than its new tokens, and where its length
    // is out of range (reported)
    int place = -1;
    if (b >= 0) {
        const int length = __ldg(a.c.kv_lens + b);
        if (cache_length(a.c, length) == length) place = length - count + (int)(t - first);
    }
    float c[8], s[8];
    const bool rotate = p.pair >= 0 && angles(a.r, a.c.T, t, place, p.pair, a.c.err, c, s);
    int64_t page = -1;
    if (place >= 0) page = page_of(a.c, b, place);
    const int in_page = place < 0 ? 0 : a.c.by_page.remainder(place);
    const int64_t slot = page * a.c.page_stride + in_page * a.c.slot_stride;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
        const int h = group + k * groups;
        const bool query = h < a.heads, value = h >= a.heads + G;
        const int g = value ? h - a.heads - G : h - a.heads;
        float x[16];
        unpack16<E>(u[k], w[k], x);
        const float* norm = query ? a.q_norm : value ? nullptr : a.k_norm;
        if (__any_sync(0xffffffffu, norm != nullptr)) {
            float y[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = x[j];
            const float* any = a.q_norm ? a.q_norm : a.k_norm;
            normalise(y, chunks, D, a.eps, (norm ? norm : any) + p.first, (norm ? norm : any) + p.second);
            if (norm) {
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = y[j];
            }
        }
        if (rotate && !value) turn(x, a.r.interleaved, c, s);
        if constexpr (H::kFormat != 0) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
            for (int o = 1; o < chunks; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (!query && h < all && page >= 0 && real) {
                float inv;
                const float scale = scale_of<H>(top, inv);
                uint8_t* dst = reinterpret_cast<uint8_t*>(value ? a.c.v : a.c.k) + slot + g * a.c.head_stride;
                *reinterpret_cast<uint2*>(dst + p.first) = make_uint2(H::encode4(x, inv), H::encode4(x + 4, inv));
                *reinterpret_cast<uint2*>(dst + p.second) =
                    make_uint2(H::encode4(x + 8, inv), H::encode4(x + 12, inv));
                if (chunk == 0)
                    (value ? a.s.v : a.s.k)[page * a.s.page_stride + g * a.s.head_stride + in_page] = scale;
            }
        } else if (!query && h < all && page >= 0 && real) {
            uint16_t* dst = (value ? a.c.v : a.c.k) + slot + g * a.c.head_stride;
            *reinterpret_cast<uint4*>(dst + p.first) = pack8<E>(x);
            *reinterpret_cast<uint4*>(dst + p.second) = pack8<E>(x + 8);
        }
        if (query && real) {
            uint16_t* dst = a.q_out + (t * a.heads + h) * D;
            *reinterpret_cast<uint4*>(dst + p.first) = pack8<E>(x);
            *reinterpret_cast<uint4*>(dst + p.second) = pack8<E>(x + 8);
        }
    }
}

// ------------------------------------------------------------------- read --

struct ReadArgs {
    CacheArgs c;
    ScaleArgs s;
    uint16_t *k, *v;  // [T, kv_heads, head_dim]
};

// 16 elements of k and of v a thread.
template <class E, class H>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs a) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (blockIdx.x == 0) check_offsets(a.c);
    const int D = a.c.head_dim, G = a.c.kv_heads, chunks = D / 16;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int chunk = (int)(i % chunks), g = (int)(i / chunks % G);
    const int64_t t = i / chunks / G;
    if (t >= a.c.T) return;
    int first, count;
    const int b = sequence_of(a.c, t, first, count);
    if (b < 0) return;
    const int length = __ldg(a.c.kv_lens + b);
    const int place = cache_length(a.c, length) == length ? length - count + (int)(t - first) : -1;
    const int64_t page = place >= 0 ? page_of(a.c, b, place) : -1;
    const int in_page = place < 0 ? 0 : a.c.by_page.remainder(place);
    const int64_t from = page * a.c.page_stride + in_page * a.c.slot_stride + g * a.c.head_stride + chunk * 16;
    const int64_t scale = page * a.s.page_stride + g * a.s.head_stride + in_page;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
        if (page >= 0) {
            if constexpr (H::kFormat == 0) {
                const uint4* src = reinterpret_cast<const uint4*>((n ? a.c.v : a.c.k) + from);
                lo = src[0];
                hi = src[1];
            } else {
                const uint4 q = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(n ? a.c.v : a.c.k) + from);
                const float s = (n ? a.s.v : a.s.k)[scale];
                float x[16];
                H::decode4(q.x, x);
                H::decode4(q.y, x + 4);
                H::decode4(q.z, x + 8);
                H::decode4(q.w, x + 12);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] *= s;
                lo = pack8<E>(x);
                hi = pack8<E>(x + 8);
            }
        }
        uint4* dst = reinterpret_cast<uint4*>((n ? a.v : a.k) + (t * G + g) * D + chunk * 16);
        dst[0] = lo;
        dst[1] = hi;
    }
}

// ------------------------------------------------------------------- host --

w4a16_status blocks_for(int64_t threads, unsigned& blocks) {
    const int64_t n = (threads + kThreads - 1) / kThreads;
    if (n > 0x7fffffffLL) return W4A16_ERR_UNSUPPORTED;
    blocks = (unsigned)n;
    return W4A16_OK;
}

// Four heads to a thread once that still leaves every SM several blocks.
bool wide(const DeviceInfo& dev, int64_t T, int64_t heads, int lanes) {
    return T * ((heads + 3) / 4) * lanes >= (int64_t)dev.sms * 4 * kThreads;
}

template <class E>
w4a16_status rope_norm(bool four, unsigned blocks, const NormArgs& a, cudaStream_t st) {
    return launch_overlapped("rope", four ? rope_norm_kernel<E, 4> : rope_norm_kernel<E, 1>, dim3(blocks), kThreads, 0,
                             st, a);
}

template <class E, class H>
w4a16_status append(bool four, unsigned blocks, const AppendArgs& a, cudaStream_t st) {
    return launch_overlapped("kv_append", four ? append_ex_kernel<E, H, 4> : append_ex_kernel<E, H, 1>, dim3(blocks),
                             kThreads, 0, st, a);
}

template <class E, class H>
w4a16_status read(unsigned blocks, const ReadArgs& a, cudaStream_t st) {
    return launch_overlapped("kv_read", read_kernel<E, H>, dim3(blocks), kThreads, 0, st, a);
}

}  // namespace

w4a16_status rope_norm_launch(const DeviceInfo& dev, int dtype, const uint16_t* x, int64_t x_row_stride,
                              int64_t x_head_stride, uint16_t* out, int64_t out_row_stride, int64_t out_head_stride,
                              int64_t T, int heads, int head_dim, const float* weight, float eps,
                              const w4a16_rotary* rotary, cudaStream_t st) {
    NormArgs a{};
    a.x = x;
    a.x_row_stride = x_row_stride;
    a.x_head_stride = x_head_stride;
    a.out = out;
    a.out_row_stride = out_row_stride;
    a.out_head_stride = out_head_stride;
    a.T = T;
    a.heads = heads;
    a.head_dim = head_dim;
    a.lanes = 1;
    while (a.lanes * 16 < head_dim) a.lanes *= 2;
    a.weight = weight;
    a.eps = eps;
    a.err = dev.error_word;
    fill(a.r, rotary);
    const bool four = wide(dev, T, heads, a.lanes);
    unsigned blocks;
    const w4a16_status s = blocks_for(T * (four ? (heads + 3) / 4 : heads) * a.lanes, blocks);
    if (s != W4A16_OK) return s;
    return dtype == W4A16_DTYPE_F16 ? rope_norm<Fp16>(four, blocks, a, st) : rope_norm<Bf16>(four, blocks, a, st);
}

w4a16_status append_ex_launch(const DeviceInfo& dev, int dtype, int format, const CacheArgs& c, const ScaleArgs& scales,
                              const uint16_t* q, int64_t q_row_stride, int64_t q_head_stride, int heads,
                              uint16_t* q_out, const uint16_t* k, int64_t k_row_stride, int64_t k_head_stride,
                              const uint16_t* v, int64_t v_row_stride, int64_t v_head_stride,
                              const w4a16_head_norms* norms, const w4a16_rotary* rotary, cudaStream_t st) {
    AppendArgs a{};
    a.c = c;
    a.s = scales;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_row_stride = q_row_stride;
    a.q_head_stride = q_head_stride;
    a.k_row_stride = k_row_stride;
    a.k_head_stride = k_head_stride;
    a.v_row_stride = v_row_stride;
    a.v_head_stride = v_head_stride;
    a.q_out = q_out;
    a.heads = q ? heads : 0;
    a.q_norm = norms && a.heads ? norms->q : nullptr;
    a.k_norm = norms ? norms->k : nullptr;
    a.eps = norms ? norms->eps : 0.0f;
    fill(a.r, rotary);
    const int64_t all = a.heads + 2 * (int64_t)c.kv_heads;
    const int lanes = c.head_dim / 16;
    const bool four = wide(dev, c.T, all, lanes);
    unsigned blocks;
    const w4a16_status s = blocks_for(c.T * (four ? (all + 3) / 4 : all) * lanes, blocks);
    if (s != W4A16_OK) return s;
    const bool f16 = dtype == W4A16_DTYPE_F16;
    switch (format) {
        case W4A16_CACHE_INT8:
            return f16 ? append<Fp16, HeldInt8>(four, blocks, a, st) : append<Bf16, HeldInt8>(four, blocks, a, st);
        case W4A16_CACHE_E4M3:
            return f16 ? append<Fp16, HeldE4m3>(four, blocks, a, st) : append<Bf16, HeldE4m3>(four, blocks, a, st);
        default:
            return f16 ? append<Fp16, Held16>(four, blocks, a, st) : append<Bf16, Held16>(four, blocks, a, st);
    }
}

w4a16_status read_launch(const DeviceInfo& dev, int dtype, int format, const CacheArgs& c, const ScaleArgs& scales,
                         uint16_t* k, uint16_t* v, cudaStream_t st) {
    ReadArgs a{};
    a.c = c;
    a.s = scales;
    a.k = k;
    a.v = v;
    unsigned blocks;
    const w4a16_status s = blocks_for(c.T * c.kv_heads * (c.head_dim / 16), blocks);
    if (s != W4A16_OK) return s;
    const bool f16 = dtype == W4A16_DTYPE_F16;
    switch (format) {
        case W4A16_CACHE_INT8: return f16 ? read<Fp16, HeldInt8>(blocks, a, st) : read<Bf16, HeldInt8>(blocks, a, st);
        case W4A16_CACHE_E4M3: return f16 ? read<Fp16, HeldE4m3>(blocks, a, st) : read<Bf16, HeldE4m3>(blocks, a, st);
        default: return f16 ? read<Fp16, Held16>(blocks, a, st) : read<Bf16, Held16>(blocks, a, st);
    }
}

}  // namespace w4a16
