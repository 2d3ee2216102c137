// Norms of the query and key heads with the position rotation in the same
// pass, the paged cache in 8 bits as it is appended to, and reading it back.
//
// A head x becomes  y = turn(x / sqrt(mean(x^2) + eps) * w)  and, in an 8-bit cache, a
// scale s and q = y / s (cache8.cuh), all in fp32 from the 16-bit input to the one rounding of
// the result. mean(x^2) and the largest |y| are over the head's 4 to 32 threads,
// of 16 elements each, by shuffles: their order is fixed.
//
// They move bytes, and the arithmetic is not far behind: some 200 instructions for 32 lanes of a
// query head, 300 of a key's (issue slots 54 to 67% busy). So a thread takes up to eight heads
// of a token, two of them loaded ahead, with the token's place, page and angles worked out once.
// The norm's weights are in shared memory; the scales of a page lie beside each other by
// head, [head][slot], so that the attention reads those of 4 places at once.
//
// Measured: 15360 tokens of 18 heads of 128 in bf16, normed and half turned by 3 axes, 146 MB: 32.0 us,
// 4.5 TB/s, 67% of the copy rate (28.7 without a norm and wholly turned); 9764 tokens of 40
// query and 8 cached heads into e4m3, 266 MB: 53.2 us, 5.0 TB/s, 74%, and into 16 bits, 280 MB: 52 us;
// reading 30011 places of 8 heads back from int8, 186 MB: 33 us, 5.7 TB/s, 85%; one token
// appended 2.8 us (a call among others in a graph).
#include <type_traits>

#include "cache8.cuh"
#include "rotary.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 3;
constexpr int kMostHeads = 8;  // of a token, to a thread
constexpr int kMostWeights = 512;

// Which heads a thread takes: `lanes` neighbours (a power of two) share `each` heads of a token. A thread block has the
// same heads (blockIdx.y) of neighbouring tokens: queries, keys and values take different paths, and warps
// that hold all three walk them all (9764 tokens of 56 heads: 84 us, and 63 so).
struct Split {
    int32_t shift, each;  // lanes = 1 << shift
    __device__ __forceinline__ int lane() const { return threadIdx.x & ((1 << shift) - 1); }
    __device__ __forceinline__ int64_t token() const {
        return (int64_t)blockIdx.x * (kThreads >> shift) + (threadIdx.x >> shift);
    }
    __device__ __forceinline__ int head() const { return blockIdx.y * each; }
};

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

// Heads are worked on twice: as they are, and once more those (of bf16) whose squares leave 32 bits. The second
// time the lanes of a head may be alone; x is multiplied by a power of two.
using Once = std::false_type;
using Again = std::true_type;

// mean(x^2) + eps over the `lanes` lanes of a head, which are among those of `mask`.
__device__ __forceinline__ float mean_square(const float (&x)[16], int lanes, unsigned mask, float mean, float eps) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += x[i] * x[i];
    for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor_sync(mask, sum, o);
    return sum * mean + eps;
}

// Whether a mean square is one that the squares it came from are held in (it is not where an element passes 2^59, or
// all and eps are as small as 2^-80).
__device__ __forceinline__ bool in_range(float square) { return square < INFINITY && square >= 8.2718061255302767e-25f; }

// x and eps times a power of two that takes their squares into range.
__device__ __forceinline__ void into_range(float (&x)[16], float& eps, float square) {
    const float f = square < 1.0f ? 1.2379400392853803e27f : 8.4703294725430034e-22f;  // 2^90, 2^-70
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= f;
    eps = eps * f * f;
}

// The lanes of the thread's head in its warp.
__device__ __forceinline__ unsigned head_mask(int lanes) {
    return (0xffffffffu >> (32 - lanes)) << (threadIdx.x & 31 & -lanes);
}

// x times r and the weights of the thread's two pieces. (In shared memory: the 16 registers that they would take
// through the loop over heads are spilled.)
__device__ __forceinline__ void weigh(float (&x)[16], float r, const float* w0, const float* w1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = *(reinterpret_cast<const float4*>(i < 2 ? w0 : w1) + (i & 1));
        x[4 * i] *= r * v.x;
        x[4 * i + 1] *= r * v.y;
        x[4 * i + 2] *= r * v.z;
        x[4 * i + 3] *= r * v.w;
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
    int32_t heads, head_dim;
    Split split;
    const float* weight;
    float eps, mean;  // mean: 1 / head_dim
    unsigned int* err;
    RotaryArgs r;
};

template <class E>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) rope_norm_kernel(const __grid_constant__ NormArgs a) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int chunk = a.split.lane();
    const int64_t t = a.split.token();
    // the lanes of a head, and those past its end, stay together for the sums
    const bool mine = t < a.T && chunk < a.head_dim / 16;
    const Pieces p = pieces_of(a.r, mine ? chunk : 0);
    const int first = a.split.head(), end = min(first + a.split.each, a.heads);
    const int real_end = mine ? end : first;
    const uint16_t* src = a.x + t * a.x_row_stride;
    auto load = [&](int h, uint4& u, uint4& w) {
        u = w = make_uint4(0, 0, 0, 0);
        if (h >= real_end) return;
        u = *reinterpret_cast<const uint4*>(src + h * a.x_head_stride + p.first);
        w = *reinterpret_cast<const uint4*>(src + h * a.x_head_stride + p.second);
    };
    uint4 u0, w0, u1, w1;
    load(first, u0, w0);
    load(first + 1, u1, w1);
    __shared__ __align__(16) float s_weight[kMostWeights];
    for (int i = threadIdx.x; i < a.head_dim; i += kThreads) s_weight[i] = __ldg(a.weight + i);
    float c[8], s[8];
    const bool rotate = mine && p.pair >= 0 && angles(a.r, a.T, t, 0, p.pair, a.err, c, s);
    __syncthreads();
    uint16_t* dst = a.out + t * a.out_row_stride;
    const int lanes = 1 << a.split.shift;
    unsigned left = 0;  // heads to be worked on again, a bit each
    auto head = [&](int h, uint4& u, uint4& w, auto again) {
        constexpr bool kAgain = decltype(again)::value;
        const unsigned mask = kAgain ? head_mask(lanes) : 0xffffffffu;
        float x[16];
        unpack16<E>(u, w, x);
        load(kAgain ? h + 1 : h + 2, u, w);
        const int bit = (h - first) & 31;
        if (kAgain && !(left >> bit & 1)) return;
        float square = mean_square(x, lanes, mask, a.mean, a.eps);
        bool done = true;
        if constexpr (kAgain) {
            if (in_range(square)) return;  // (another head of the bit, of more than 32)
            float eps = a.eps;
            into_range(x, eps, square);
            square = mean_square(x, lanes, mask, a.mean, eps);
        } else {
            done = in_range(square);
            left |= (done ? 0u : 1u) << bit;
        }
        weigh(x, rsqrtf(square), s_weight + p.first, s_weight + p.second);
        if (rotate) turn(x, a.r.interleaved, c, s);
        if (h >= real_end || !done) return;
        *reinterpret_cast<uint4*>(dst + h * a.out_head_stride + p.first) = pack8<E>(x);
        *reinterpret_cast<uint4*>(dst + h * a.out_head_stride + p.second) = pack8<E>(x + 8);
    };
#pragma unroll 1
    for (int h = first; h < end; h += 2) {
        head(h, u0, w0, Once{});
        if (h + 1 < end) head(h + 1, u1, w1, Once{});
    }
    if (!left) return;
    load(first, u0, w0);
#pragma unroll 1
    for (int h = first; h < end; ++h) head(h, u0, w0, Again{});
}

// ----------------------------------------------------------------- append --

struct AppendArgs {
    CacheArgs c;
    ScaleArgs s;
    const uint16_t *q, *k, *v;
    int64_t q_row_stride, q_head_stride, k_row_stride, k_head_stride, v_row_stride, v_head_stride;
    uint16_t* q_out;  // [T, heads, head_dim]
    int32_t heads;    // 0: no q
    Split split;
    const float *q_norm, *k_norm;  // nullptr: left as they are
    float eps, mean;               // mean: 1 / head_dim
    RotaryArgs r;
};

// The heads of a token in one row: queries, then keys, then values.
template <class E, class H>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) append_ex_kernel(const __grid_constant__ AppendArgs a) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(a.c);
    const int D = a.c.head_dim, G = a.c.kv_heads;
    const int chunks = D / 16;  // 4 or 8
    const int all = a.heads + 2 * G;
    const int chunk = a.split.lane();
    int64_t t = a.split.token();
    const bool real = t < a.c.T;  // lanes without a token stay for the sums
    if (!real) t = a.c.T - 1;
    const Pieces p = pieces_of(a.r, chunk);
    const int begin = a.split.head(), end = min(begin + a.split.each, all);
    const int real_end = real ? end : begin;
    auto load = [&](int h, uint4& u, uint4& w) {
        u = w = make_uint4(0, 0, 0, 0);
        if (h >= real_end) return;
        const uint16_t* src = h < a.heads ? a.q + t * a.q_row_stride + h * a.q_head_stride
                              : h < a.heads + G ? a.k + t * a.k_row_stride + (h - a.heads) * a.k_head_stride
                                                : a.v + t * a.v_row_stride + (h - a.heads - G) * a.v_head_stride;
        u = *reinterpret_cast<const uint4*>(src + p.first);
        w = *reinterpret_cast<const uint4*>(src + p.second);
    };
    uint4 u0, w0, u1, w1;
    load(begin, u0, w0);
    load(begin + 1, u1, w1);
    __shared__ __align__(16) float s_weight[2][128];  // queries', keys'
    if (a.q_norm && threadIdx.x < D) s_weight[0][threadIdx.x] = __ldg(a.q_norm + threadIdx.x);
    if (a.k_norm && threadIdx.x < D) s_weight[1][threadIdx.x] = __ldg(a.k_norm + threadIdx.x);
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
    const int64_t scale_slot = page * a.s.page_stride + in_page;
    __syncthreads();
    unsigned left = 0;  // heads to be worked on again, a bit each
    auto head = [&](int h, uint4& u, uint4& w, auto again) {  // (h is that of the whole thread block)
        constexpr bool kAgain = decltype(again)::value;
        const unsigned mask = kAgain ? head_mask(chunks) : 0xffffffffu;
        const bool query = h < a.heads, value = h >= a.heads + G;
        const int g = value ? h - a.heads - G : h - a.heads;
        float x[16];
        unpack16<E>(u, w, x);
        load(kAgain ? h + 1 : h + 2, u, w);
        const int bit = (h - begin) & 31;
        if (kAgain && !(left >> bit & 1)) return;
        bool done = true;
        if (query ? a.q_norm != nullptr : !value && a.k_norm != nullptr) {
            float square = mean_square(x, chunks, mask, a.mean, a.eps);
            if constexpr (kAgain) {
                if (in_range(square)) return;  // (another head of the bit, of more than 32)
                float eps = a.eps;
                into_range(x, eps, square);
                square = mean_square(x, chunks, mask, a.mean, eps);
            } else {
                done = in_range(square);
                left |= (done ? 0u : 1u) << bit;
            }
            weigh(x, rsqrtf(square), s_weight[!query] + p.first, s_weight[!query] + p.second);
        }
        if (rotate && !value) turn(x, a.r.interleaved, c, s);
        float top = 0.0f;
        if constexpr (H::kFormat != 0) {
            if (!query) {
#pragma unroll
                for (int j = 0; j < 16; ++j) top = max_nan(top, fabsf(x[j]));
                for (int o = 1; o < chunks; o <<= 1) top = max_nan(top, __shfl_xor_sync(mask, top, o));
            }
        }
        if (h >= real_end || !done) return;
        if (query) {
            uint16_t* dst = a.q_out + (t * a.heads + h) * D;
            *reinterpret_cast<uint4*>(dst + p.first) = pack8<E>(x);
            *reinterpret_cast<uint4*>(dst + p.second) = pack8<E>(x + 8);
        } else if (page >= 0) {
            if constexpr (H::kFormat != 0) {
                float inv;
                const float scale = scale_of<H>(top, inv);
                uint8_t* dst = reinterpret_cast<uint8_t*>(value ? a.c.v : a.c.k) + slot + g * a.c.head_stride;
                *reinterpret_cast<uint2*>(dst + p.first) = make_uint2(H::encode4(x, inv), H::encode4(x + 4, inv));
                *reinterpret_cast<uint2*>(dst + p.second) =
                    make_uint2(H::encode4(x + 8, inv), H::encode4(x + 12, inv));
                if (chunk == 0) (value ? a.s.v : a.s.k)[scale_slot + g * a.s.head_stride] = scale;
            } else {
                uint16_t* dst = (value ? a.c.v : a.c.k) + slot + g * a.c.head_stride;
                *reinterpret_cast<uint4*>(dst + p.first) = pack8<E>(x);
                *reinterpret_cast<uint4*>(dst + p.second) = pack8<E>(x + 8);
            }
        }
    };
#pragma unroll 1
    for (int h = begin; h < end; h += 2) {
        head(h, u0, w0, Once{});
        __syncwarp();
        if (h + 1 < end) head(h + 1, u1, w1, Once{});
        __syncwarp();
    }
    if (!left) return;
    load(begin, u0, w0);
#pragma unroll 1
    for (int h = begin; h < end; ++h) head(h, u0, w0, Again{});
}

// ------------------------------------------------------------------- read --

struct ReadArgs {
    CacheArgs c;
    ScaleArgs s;
    int32_t shift;      // 1 << shift lanes to a head
    FastDiv by_heads;   // of T * kv_heads,
    int32_t few;        // if they are fewer than 2^31
    uint16_t *k, *v;    // [T, kv_heads, head_dim]
};

// 16 elements of k and of v a thread, the heads of a token side by side (their rows are, in the result).
template <class E, class H>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs a) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (blockIdx.x == 0) check_offsets(a.c);
    const int D = a.c.head_dim, G = a.c.kv_heads;
    const int chunk = threadIdx.x & ((1 << a.shift) - 1);
    const int64_t row = (int64_t)blockIdx.x * (kThreads >> a.shift) + (threadIdx.x >> a.shift);
    const int64_t t = a.few ? a.by_heads.quotient((int)row) : row / G;  // (a division in 64 bits: 60 instructions)
    const int g = (int)(row - t * G);
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
                const uint8_t* src = reinterpret_cast<const uint8_t*>(n ? a.c.v : a.c.k) + from;
                const uint4 q = *reinterpret_cast<const uint4*>(src);
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

// The split of T tokens' heads of `chunks` 16-element pieces, and its thread blocks: as many heads to a thread as leave
// every SM two rounds of blocks (what depends on the token is worked out once a thread), `most` at most.
w4a16_status split_for(const DeviceInfo& dev, int64_t T, int64_t heads, int chunks, int most, Split& s,
                       dim3& grid) {
    s.shift = 0;
    while ((1 << s.shift) < chunks) ++s.shift;
    const int64_t per = kThreads >> s.shift, n = (T + per - 1) / per;
    int64_t each = n * heads / (dev.sms * kBlocksPerSm * 2);
    each = each > most ? most : each;
    const int64_t least = (heads + 65534) / 65535;  // what a grid's second dimension takes
    each = each < least ? least : each;
    int64_t groups = (heads + each - 1) / each;
    each = (heads + groups - 1) / groups;
    groups = (heads + each - 1) / each;
    if (n > 0x7fffffffLL) return W4A16_ERR_UNSUPPORTED;
    s.each = (int)each;
    grid = dim3((unsigned)n, (unsigned)groups);
    return W4A16_OK;
}

template <class E>
w4a16_status rope_norm(const dim3& grid, const NormArgs& a, cudaStream_t st) {
    return launch_overlapped("rope", rope_norm_kernel<E>, grid, kThreads, 0, st, a);
}

template <class E, class H>
w4a16_status append(const dim3& grid, const AppendArgs& a, cudaStream_t st) {
    return launch_overlapped("kv_append", append_ex_kernel<E, H>, grid, kThreads, 0, st, a);
}

template <class E, class H>
w4a16_status read(const dim3& grid, const ReadArgs& a, cudaStream_t st) {
    return launch_overlapped("kv_read", read_kernel<E, H>, grid, kThreads, 0, st, a);
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
    a.weight = weight;
    a.eps = eps;
    a.mean = 1.0f / (float)head_dim;
    a.err = dev.error_word;
    fill(a.r, rotary);
    dim3 grid;
    const w4a16_status s = split_for(dev, T, heads, head_dim / 16, kMostHeads, a.split, grid);
    if (s != W4A16_OK) return s;
    return dtype == W4A16_DTYPE_F16 ? rope_norm<Fp16>(grid, a, st) : rope_norm<Bf16>(grid, a, st);
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
    a.mean = 1.0f / (float)c.head_dim;
    fill(a.r, rotary);
    dim3 grid;
    const w4a16_status s = split_for(dev, c.T, a.heads + 2 * (int64_t)c.kv_heads, c.head_dim / 16, kMostHeads,
                                     a.split, grid);
    if (s != W4A16_OK) return s;
    const bool f16 = dtype == W4A16_DTYPE_F16;
    switch (format) {
        case W4A16_CACHE_INT8:
            return f16 ? append<Fp16, HeldInt8>(grid, a, st) : append<Bf16, HeldInt8>(grid, a, st);
        case W4A16_CACHE_E4M3:
            return f16 ? append<Fp16, HeldE4m3>(grid, a, st) : append<Bf16, HeldE4m3>(grid, a, st);
        default:
            return f16 ? append<Fp16, Held16>(grid, a, st) : append<Bf16, Held16>(grid, a, st);
    }
}

w4a16_status read_launch(const DeviceInfo&, int dtype, int format, const CacheArgs& c, const ScaleArgs& scales,
                         uint16_t* k, uint16_t* v, cudaStream_t st) {
    ReadArgs a{};
    a.c = c;
    a.s = scales;
    a.k = k;
    a.v = v;
    a.shift = c.head_dim == 128 ? 3 : 2;
    const int64_t per = kThreads >> a.shift, blocks = (c.T * c.kv_heads + per - 1) / per;
    if (blocks > 0x7fffffffLL) return W4A16_ERR_UNSUPPORTED;
    a.by_heads = fast_div(c.kv_heads);
    a.few = blocks * per < 0x7fffffffLL;
    const dim3 grid((unsigned)blocks);
    const bool f16 = dtype == W4A16_DTYPE_F16;
    switch (format) {
        case W4A16_CACHE_INT8: return f16 ? read<Fp16, HeldInt8>(grid, a, st) : read<Bf16, HeldInt8>(grid, a, st);
        case W4A16_CACHE_E4M3: return f16 ? read<Fp16, HeldE4m3>(grid, a, st) : read<Bf16, HeldE4m3>(grid, a, st);
        default: return f16 ? read<Fp16, Held16>(grid, a, st) : read<Bf16, Held16>(grid, a, st);
    }
}

}  // namespace w4a16
