// Rotary positions, and appending keys and values to a paged cache with the
// rotation applied on the way.
//
// A pair (a, b) of a head turns by the angle of its position p on its axis:
//     (a, b) -> (a cos - b sin, b cos + a sin),   cos, sin = table[p, pair]
// in fp32, rounded once to the element type. The angles come from a table (made
// once, in 64 bits: fp32 arithmetic on the angle itself would lose position
// 10^6 in its last bits), one row of rotary_dim floats per position. Pairs are
// elements (i, i + rotary_dim / 2) or, interleaved, (2i, 2i + 1); elements past
// rotary_dim are copied. With several axes each pair reads the row of its own
// axis's position.
//
// Both kernels move bytes and do little else. A thread takes the 16 elements
// of 8 pairs: two 16-byte pieces that are 8 lanes wide each, so a head's row
// is read and written in whole 128-byte lines. It keeps its 8 cosines and
// sines in registers for HPT heads of the same token and issues all their
// loads before the first store.
#include "attention.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;  // rotary_dim <= 256

struct RotaryArgs {
    const float* table;       // [rows, dim], cos of the pairs and then sin; nullptr: no rotation
    int64_t rows;
    int32_t dim, interleaved;
    const int32_t* positions;  // [axes, T], nullptr: the place in the sequence
    int32_t axes;
    uint8_t pair_axis[kMaxPairs];
};

// The element pieces of thread-chunk `chunk` of a head: 8 pairs, or 16
// consecutive elements past the rotary width.
struct Pieces {
    int first, second;  // element offsets of the two 16-byte pieces
    int pair;           // first pair, or -1 for a plain copy
};

__device__ __forceinline__ Pieces pieces_of(const RotaryArgs& r, int chunk) {
    Pieces p;
    const int turned = r.table ? r.dim / 16 : 0;
    if (chunk >= turned) {
        p.first = chunk * 16;
        p.second = p.first + 8;
        p.pair = -1;
    } else {
        p.pair = chunk * 8;
        p.first = r.interleaved ? chunk * 16 : chunk * 8;
        p.second = r.interleaved ? p.first + 8 : p.first + r.dim / 2;
    }
    return p;
}

// Cosines and sines of 8 pairs of token t. `place` is the position used when
// the caller gave none. Returns false (nothing to turn) where there is no such
// position. One outside the table is reported, and the pairs of its axis turn by
// nothing: false, or a cosine of 1 among pairs of other axes.
__device__ __forceinline__ bool angles(const RotaryArgs& r, int64_t T, int64_t t, int place, int pair,
                                       unsigned int* err, float (&c)[8], float (&s)[8]) {
    const int half = r.dim / 2;
    int pos[8];
    bool same = true;
    if (!r.positions) {
        if (place < 0) return false;
#pragma unroll
        for (int i = 0; i < 8; ++i) pos[i] = place;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            pos[i] = __ldg(r.positions + r.pair_axis[pair + i] * T + t);
            same = same && r.pair_axis[pair + i] == r.pair_axis[pair];
        }
    }
    bool ok = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) ok = ok && pos[i] >= 0 && pos[i] < r.rows;
    if (!ok) {
        raise_device_error(err, W4A16_ERR_BAD_CACHE);
        if (same || r.rows == 0) return false;
    }
    if (same) {
        const float4* row = reinterpret_cast<const float4*>(r.table + (int64_t)pos[0] * r.dim + pair);
        const float4* row_s = reinterpret_cast<const float4*>(r.table + (int64_t)pos[0] * r.dim + half + pair);
        const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(row_s), s1 = __ldg(row_s + 1);
        c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
        c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
        s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
        s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
    } else {
        // from the last row for a position outside (as from a negative one), and put right below: a
        // test at each load costs the append of 3 axes 7%
        const uint32_t last = (uint32_t)min(r.rows - 1, (int64_t)0x7fffffff);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float* row = r.table + (int64_t)min((uint32_t)pos[i], last) * r.dim + pair + i;
            c[i] = __ldg(row);
            s[i] = __ldg(row + half);
        }
        if (!ok) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int p = __ldg(r.positions + r.pair_axis[pair + i] * T + t);
                if (p < 0 || p >= r.rows) {
                    c[i] = 1.0f;
                    s[i] = 0.0f;
                }
            }
        }
    }
    return true;
}

// Turns the 8 pairs held in two 16-byte pieces.
template <class E>
__device__ __forceinline__ void turn(uint4& u, uint4& w, bool interleaved, const float (&c)[8], const float (&s)[8]) {
    uint32_t x[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = E::unpack(x[i]);
            x[i] = E::pack(v.x * c[i] - v.y * s[i], v.y * c[i] + v.x * s[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = E::unpack(x[i]), b = E::unpack(x[i + 4]);
            x[i] = E::pack(a.x * c[2 * i] - b.x * s[2 * i], a.y * c[2 * i + 1] - b.y * s[2 * i + 1]);
            x[i + 4] = E::pack(b.x * c[2 * i] + a.x * s[2 * i], b.y * c[2 * i + 1] + a.y * s[2 * i + 1]);
        }
    }
    u = make_uint4(x[0], x[1], x[2], x[3]);
    w = make_uint4(x[4], x[5], x[6], x[7]);
}

// ------------------------------------------------------------------- rope --

struct RopeArgs {
    const uint16_t* x;
    int64_t x_row_stride, x_head_stride;
    uint16_t* out;
    int64_t out_row_stride, out_head_stride;
    int64_t T;
    int32_t heads, head_dim;
    unsigned int* err;
    RotaryArgs r;
};

template <class E, int HPT>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int chunks = a.head_dim / 16;
    const int groups = (a.heads + HPT - 1) / HPT;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int chunk = (int)(i % chunks);
    const int group = (int)(i / chunks % groups);
    const int64_t t = i / chunks / groups;
    if (t >= a.T) return;
    const Pieces p = pieces_of(a.r, chunk);
    uint4 u[HPT], w[HPT];
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
        const int h = group + k * groups;
        if (h >= a.heads) continue;
        const uint16_t* src = a.x + t * a.x_row_stride + h * a.x_head_stride;
        u[k] = *reinterpret_cast<const uint4*>(src + p.first);
        w[k] = *reinterpret_cast<const uint4*>(src + p.second);
    }
    float c[8], s[8];
    const bool rotate = p.pair >= 0 && angles(a.r, a.T, t, 0, p.pair, a.err, c, s);
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
        const int h = group + k * groups;
        if (h >= a.heads) continue;
        if (rotate) turn<E>(u[k], w[k], a.r.interleaved, c, s);
        uint16_t* dst = a.out + t * a.out_row_stride + h * a.out_head_stride;
        *reinterpret_cast<uint4*>(dst + p.first) = u[k];
        *reinterpret_cast<uint4*>(dst + p.second) = w[k];
    }
}

// ----------------------------------------------------------------- append --

struct AppendArgs {
    CacheArgs c;
    const uint16_t *q, *k, *v;
    int64_t q_row_stride, q_head_stride, k_row_stride, k_head_stride, v_row_stride, v_head_stride;
    uint16_t* q_out;  // [T, heads, head_dim]
    int32_t heads;    // 0: no q
    RotaryArgs r;
};

// The heads of a token in one row: queries, then keys, then values.
// (Five thread blocks an SM with one head a thread: left to itself the compiler takes registers for the rare path.)
template <class E, int HPT>
__global__ void __launch_bounds__(kThreads, HPT == 1 ? 5 : 3) append_kernel(const __grid_constant__ AppendArgs a) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (blockIdx.x == 0) check_offsets(a.c);
    const int D = a.c.head_dim, G = a.c.kv_heads;
    const int chunks = D / 16;
    const int all = a.heads + 2 * G;
    const int groups = (all + HPT - 1) / HPT;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int chunk = (int)(i % chunks);
    const int group = (int)(i / chunks % groups);
    const int64_t t = i / chunks / groups;
    if (t >= a.c.T) return;
    const Pieces p = pieces_of(a.r, chunk);
    uint4 u[HPT], w[HPT];
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
        const int h = group + k * groups;
        if (h >= all) continue;
        const uint16_t* src = h < a.heads ? a.q + t * a.q_row_stride + h * a.q_head_stride
                              : h < a.heads + G ? a.k + t * a.k_row_stride + (h - a.heads) * a.k_head_stride
                                                : a.v + t * a.v_row_stride + (h - a.heads - G) * a.v_head_stride;
        u[k] = *reinterpret_cast<const uint4*>(src + p.first);
        w[k] = *reinterpret_cast<const uint4*>(src + p.second);
    }
    int first, count;
    const int b = sequence_of(a.c, t, first, count);
    // place in the sequence; negative where the sequence is shorter than its new tokens, and where its length
    // is out of range (reported): held to the range, that one would name places that are taken
    int place = -1;
    if (b >= 0) {
        const int length = __ldg(a.c.kv_lens + b);
        if (cache_length(a.c, length) == length) place = length - count + (int)(t - first);
    }
    float c[8], s[8];
    const bool rotate = p.pair >= 0 && angles(a.r, a.c.T, t, place, p.pair, a.c.err, c, s);
    int64_t page = -1;
    if (place >= 0) page = page_of(a.c, b, place);
    const int64_t slot = page * a.c.page_stride + (place < 0 ? 0 : a.c.by_page.remainder(place)) * a.c.slot_stride;
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
        const int h = group + k * groups;
        if (h >= all) continue;
        const bool value = h >= a.heads + G;
        if (rotate && !value) turn<E>(u[k], w[k], a.r.interleaved, c, s);
        uint16_t* dst;
        if (h < a.heads) {
            dst = a.q_out + (t * a.heads + h) * D;
        } else {
            if (page < 0) continue;
            dst = value ? a.c.v + slot + (h - a.heads - G) * a.c.head_stride
                        : a.c.k + slot + (h - a.heads) * a.c.head_stride;
        }
        *reinterpret_cast<uint4*>(dst + p.first) = u[k];
        *reinterpret_cast<uint4*>(dst + p.second) = w[k];
    }
}

// ------------------------------------------------------------------- host --

// Four heads to a thread once that still leaves every SM several blocks.
bool wide(const DeviceInfo& dev, int64_t T, int64_t heads, int head_dim) {
    return T * ((heads + 3) / 4) * (head_dim / 16) >= (int64_t)dev.sms * 4 * kThreads;
}

void fill(RotaryArgs& r, const w4a16_rotary* rotary) {
    r = RotaryArgs{};
    if (!rotary) return;
    r.table = rotary->table;
    r.rows = rotary->rows;
    r.dim = rotary->rotary_dim;
    r.interleaved = rotary->interleaved;
    r.positions = rotary->positions;
    r.axes = rotary->axes;
    for (int i = 0; i < rotary->rotary_dim / 2; ++i) r.pair_axis[i] = rotary->pair_axes ? rotary->pair_axes[i] : 0;
}

template <class A>
w4a16_status run(const char* what, void (*narrow)(A), void (*wide4)(A), bool four, const A& a, int64_t T, int64_t heads,
                 int head_dim, cudaStream_t st) {
    const int64_t groups = four ? (heads + 3) / 4 : heads;
    const int64_t blocks = (T * groups * (head_dim / 16) + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL) return W4A16_ERR_UNSUPPORTED;
    return launch_overlapped(what, four ? wide4 : narrow, dim3((unsigned)blocks), kThreads, 0, st, a);
}

}  // namespace

w4a16_status rope_launch(const DeviceInfo& dev, int dtype, const uint16_t* x, int64_t x_row_stride,
                         int64_t x_head_stride, uint16_t* out, int64_t out_row_stride, int64_t out_head_stride,
                         int64_t T, int heads, int head_dim, const w4a16_rotary* rotary, cudaStream_t st) {
    RopeArgs a{};
    a.x = x;
    a.x_row_stride = x_row_stride;
    a.x_head_stride = x_head_stride;
    a.out = out;
    a.out_row_stride = out_row_stride;
    a.out_head_stride = out_head_stride;
    a.T = T;
    a.heads = heads;
    a.head_dim = head_dim;
    a.err = dev.error_word;
    fill(a.r, rotary);
    const bool four = wide(dev, T, heads, head_dim);
    return dtype == W4A16_DTYPE_F16
               ? run("rope", rope_kernel<Fp16, 1>, rope_kernel<Fp16, 4>, four, a, T, heads, head_dim, st)
               : run("rope", rope_kernel<Bf16, 1>, rope_kernel<Bf16, 4>, four, a, T, heads, head_dim, st);
}

w4a16_status append_launch(const DeviceInfo& dev, int dtype, const CacheArgs& c, const uint16_t* q,
                           int64_t q_row_stride, int64_t q_head_stride, int heads, uint16_t* q_out,
                           const uint16_t* k, int64_t k_row_stride, int64_t k_head_stride, const uint16_t* v,
                           int64_t v_row_stride, int64_t v_head_stride, const w4a16_rotary* rotary,
                           cudaStream_t st) {
    AppendArgs a{};
    a.c = c;
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
    fill(a.r, rotary);
    const int64_t all = a.heads + 2 * (int64_t)c.kv_heads;
    const bool four = wide(dev, c.T, all, c.head_dim);
    return dtype == W4A16_DTYPE_F16
               ? run("kv_append", append_kernel<Fp16, 1>, append_kernel<Fp16, 4>, four, a, c.T, all, c.head_dim, st)
               : run("kv_append", append_kernel<Bf16, 1>, append_kernel<Bf16, 4>, four, a, c.T, all, c.head_dim, st);
}

}  // namespace w4a16
