// Attention over the paged cache for few rows: single tokens, and the few rows
// of draft tokens (up to 16 rows per cached head, a row being one query head
// of one new token; heads that share a cached head share its reads).
//
// out = softmax(c q k^T) v in one pass: with m the running maximum of a row's
// scores s and p_j = 2^(s_j - m), both l = sum p_j and o = sum p_j v_j are
// multiplied by 2^(m - m') when the maximum moves to m'. p is rounded to the
// element type for the second product. The maximum moves with every score
// that passes it, so the largest weight is 1 and exact, and where few weights count,
// little is lost: 1.00 to 1.07 times the error of rounding the result alone, where a
// maximum that lags (by up to 2^14 or 2^40 in p) gives 1.3 to 2.0, at the same speed.
//
// What bounds it is reading the cache once: 2 D 16-bit elements of k and v per place and
// cached head, against 4 D operations for each row. So the work is spread over
// the whole GPU by bytes, whatever the lengths are: the list of 64-place blocks of all
// (sequence, cached head) items is cut into equal runs, one per thread block, on
// the device (the lengths never come to the host). Items that a cut divides are
// joined through the workspace: each part leaves its m, l and o, and the part
// that finishes last adds them up in their order along the sequence.
//
// Within a thread block each of 4 warps takes 16 places of a 64-place block
// and keeps its own m, l and o to the end of the item; nothing but the end
// synchronizes them. k and v go through a private ring of shared memory per
// warp (cp.async, 24 KB a warp, two thread blocks an SM: 128 to 160 KB in
// flight per SM; 6.8 TB/s times 1 us of latency needs 45), across items without draining. The
// products are formed transposed, s^T = k q^T and o^T = v^T p^T, so that
// the 16-wide side of the m16n8k16 MMA is places and head elements, all of them
// real, and the rows fill the 8-wide side: one of them for up to 8 rows, two for
// 16. p reaches the second product's operand layout by an 8x8 register transpose.
//
// Over an 8-bit cache (HeldInt8, HeldE4m3) a step has half the bytes. The rows come to fp16 as they are
// held, exactly, on their way from shared memory to the products: integers by three integer
// operations and a subtraction for four, e4m3 by the hardware's conversion. A lane reads keys 16 bytes
// at a time in whatever order of elements that gives, and the queries in the same one;
// values come by the transposing load in pairs of bytes, which are two output rows. The scale
// of a key multiplies its scores and that of a value its softmax weights, both in fp32. bf16
// queries go to fp16 divided by a power of two. Up to 48 rows are taken, in groups of 16 on thread
// blocks that run side by side and read the same bytes. What bounds it is still the cache's bytes, but
// the products' preparation is close behind (issue slots 47 to 53% busy, the integer pipe 43 to
// 50%): three thread blocks an SM with 12 warps were 2% faster on short sequences and 6% slower on long ones.
//
// Measured (heads of 128, 8 cached): one token each of 64 sequences of 300 to
// 8000 places, 1.10 GB: 171 us, 6.4 TB/s, 95% of the copy rate; two of 125000
// and 133000 places, 1.06 GB: 167 us, 6.3 TB/s; one of 777 places 10 us, which is
// latency: 2 us of launch, 1 to find the run, 2 for page entries and then k and
// v, 1 for a block's products with instructions not yet cached, 4 for the join.
// Over 8 bits: 64 such sequences, 0.574 GB: 109 us, 5.3 TB/s, 79% of the copy rate; two of 120 to
// 150 thousand places in e4m3, 0.559 GB: 97 us, 5.8 TB/s, 87%; one of 777 places 10 us; 3 and 5
// tokens (15 and 25 rows) of 16 sequences of 2000 to 9000 places, 0.175 GB: 55 and 93 us, where
// reading them once is 26.
#pragma once

#include <type_traits>

#include "cache8.cuh"

namespace w4a16 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 16;               // places per warp step
constexpr int kBlock = kWarps * kStep;  // places per block of the work list
constexpr int kBlocksPerSm = 2;
constexpr int kRingBytes = 24 * 1024;   // per warp

template <class H, int D>
struct Layout {
    static constexpr bool kHeld8 = H::kFormat != 0;
    static constexpr int kRowBytes = kHeld8 ? D : D * 2;
    static constexpr int kChunks = kRowBytes / 16;              // 16-byte pieces per row
    static constexpr int kHalfStage = kStep * kRowBytes;        // k, then v, then their scales
    static constexpr int kScaleBytes = kHeld8 ? 2 * kStep * 4 : 0;
    static constexpr int kStage = 2 * kHalfStage + kScaleBytes;
    static constexpr int kStages = kRingBytes / kStage;
    static constexpr int kJoinBytes = kWarps * 8 * D * 4;
    static constexpr int kSmem = kWarps * kRingBytes + kJoinBytes;
    // piece `chunk` of row `row`; eight rows of one chunk fall into eight different bank groups
    __device__ static __forceinline__ uint32_t at(int row, int chunk) {
        if constexpr (kRowBytes == 64) return (uint32_t)(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
        return (uint32_t)(row * kRowBytes + ((chunk ^ (row & 7)) << 4));
    }
    // element d of column `col` of a warp's part of o (floats); the four column
    // pairs of a lane group fall into four different groups of 8 banks
    __device__ static __forceinline__ int join_at(int warp, int col, int d) {
        return (warp * 8 + col) * D + (d ^ ((col >> 1) << 3));
    }
};

template <class E>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (E::kDtype == W4A16_DTYPE_F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// A bf16 row of queries (row n of qf, spread over 4 lanes) in fp16, divided by the power of two of its largest
// element, which is returned: exact, but for elements below 2^-14 of the largest, which keep 2^-25 of it.
template <int KS, int NT>
__device__ __forceinline__ float to_fp16_row(uint32_t (&qf)[KS][NT][2], int n) {
    uint32_t top = 0;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int j = 0; j < 2; ++j) top = max(top, max((qf[ks][n][j] & 0x7FFFu) << 16, qf[ks][n][j] & 0x7FFF0000u));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t e = min(max(top >> 23, 1u), 253u);  // the exponent and 127
    const float down = __uint_as_float((254u - e) << 23);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 v = Bf16::unpack(qf[ks][n][j]);
            qf[ks][n][j] = Fp16::pack(v.x * down, v.y * down);
        }
    return __uint_as_float(e << 23);
}

// What the weights of the second product over an 8-bit cache are multiplied by: the largest is then at 2^14, and
// fp16 holds what is 2^-38 of it.
constexpr float kWeightUp = 16384.0f;
// What the logarithm of a value's scale is taken for if it is less (of zeros 2^-100 / most, or 0): the sum's terms are
// then at most 2^96, and 2^30 of them inside 32 bits.
constexpr float kLeastLog2 = -96.0f;

struct StepArgs {
    AttentionArgs a;
    int* counters;   // one per thread block, zero between calls
    float* parts;    // [2 * blocks][rows][D]: o of the parts of divided items
    float2* stats;   // [2 * blocks][rows]: their m and l
    // of an 8-bit cache:
    ScaleArgs s;
    int lanes, turns;  // cached heads that are worked on side by side, and how many times that makes them all
    int row_groups;    // of a head's rows, side by side too
};

// A sequence as this kernel sees it; blocks == 0: not one of its own.
struct Sequence {
    int first, count, length;
    int low;         // first place that any row sees
    int block, blocks;  // its 64-place blocks: the first, and how many (one at least, so that empty rows are written)
};

// A sequence with rows from row0 on, and no more than max_rows.
__device__ __forceinline__ void load_sequence(const AttentionArgs& a, int b, int row0, int max_rows, Sequence& s) {
    const int first = __ldg(a.c.q_offsets + b), next = __ldg(a.c.q_offsets + b + 1), length = __ldg(a.c.kv_lens + b);
    s.first = first;
    s.count = next - first;
    s.blocks = 0;
    if (first < 0 || next > a.c.T || s.count <= 0 || s.count > a.max_q_len || s.count * a.ratio > max_rows) return;
    if (s.count * a.ratio <= row0) return;
    s.length = cache_length(a.c, length);
    s.low = first_seen(a, s.length - s.count);
    s.block = s.low / kBlock;
    s.blocks = max(1, (s.length + kBlock - 1) / kBlock - s.block);
}

// Run `run` of `runs` of `total` units.
__device__ __forceinline__ void share_out(int64_t total, unsigned run, unsigned runs, Shares& shares, int64_t& begin,
                                          int64_t& end) {
    shares.base = total / runs;
    shares.more = (int)(total - shares.base * runs);
    begin = shares.start(run);
    end = shares.start(run + 1);
}

// A position in the work list, as a warp walks it.
struct Cursor {
    int b, g, block, end;  // block of the sequence, and one past the item's last
    Sequence s;
};

// turns: of the cached heads of a sequence (each, or `lanes` of them, is an item)
__device__ __forceinline__ void next_item(const AttentionArgs& a, int row0, int max_rows, int turns, Cursor& c) {
    if (++c.g == turns) {
        c.g = 0;
        do {
            if (++c.b >= a.c.batch) {  // past the list's end: never used
                c.s.blocks = 0;
                break;
            }
            load_sequence(a, c.b, row0, max_rows, c.s);
        } while (c.s.blocks == 0);
    }
    c.block = c.s.block;
    c.end = c.s.block + c.s.blocks;
}

template <class E, class H, int D, int NT>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) step_kernel(const __grid_constant__ StepArgs arg) {
    using L = Layout<H, D>;
    constexpr bool kHeld8 = L::kHeld8;
    using M = std::conditional_t<kHeld8, Fp16, E>;  // of the products
    constexpr int kOutChunks = D / 8;               // threads to a row of the result
    constexpr int kRows = NT * 8;
    constexpr int kKs = D / 16;  // k-steps of the scores; 16-element tiles of the output
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t s_sum[kWarps];
    __shared__ int s_found[2];
    __shared__ float2 s_stats[kWarps][kRows];
    __shared__ int s_last;
    const AttentionArgs& a = arg.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int grp = lane >> 2, quad = lane & 3;
    const int ratio = a.ratio;
    // Over an 8-bit cache a run of blocks is that of `lanes` thread blocks, a cached head each: the rows of a place's
    // heads are neighbours in memory, and so are read at the same time. (With runs of one head after another, whose
    // 128 bytes of a place are read alone, 64 sequences took 119 us and two long ones 118, where these runs
    // took 113 and 106 with three thread blocks an SM; 127 and 111, 118 and 101 with two.)
    // Of more rows than one thread block takes, groups of them go side by side as well.
    const int lanes = kHeld8 ? arg.lanes : 1, turns = kHeld8 ? arg.turns : a.c.kv_heads;
    const int side = kHeld8 ? lanes * arg.row_groups : 1, max_rows = kHeld8 ? kRows * arg.row_groups : kRows;
    const unsigned run = blockIdx.x / side, runs = gridDim.x / side;
    const int member = kHeld8 ? (int)(blockIdx.x - run * side) : 0;
    const int head0 = kHeld8 ? member % lanes : 0, row0 = kHeld8 ? member / lanes * kRows : 0;
    // A sum to the maximum m brought to the larger one `top` (a sum of NaN stays one).
    auto rescaled = [](float sum, float m, float top) {
        const float d = m == -INFINITY ? m : m - top;
        return kHeld8 ? times_exp2(sum, d) : sum * fast_exp2(d);
    };
    auto head_of = [&](int g) { return kHeld8 ? min(g * lanes + head0, a.c.kv_heads - 1) : g; };

    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (blockIdx.x == 0) check_offsets(a.c);
    if (kHeld8 && run >= runs) return;

    // the length of the work list, then the item in which this thread block's
    // run starts; one round does for both while there are no more sequences than threads
    Shares shares;
    int64_t run_begin = 0, run_end = 0;
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
        int64_t before = 0;
#pragma unroll 1
        for (int b0 = 0; b0 < a.c.batch; b0 += kThreads) {
            Sequence s;
            int64_t n = 0;
            if (b0 + tid < a.c.batch) {
                load_sequence(a, b0 + tid, row0, max_rows, s);
                n = (int64_t)s.blocks * turns;
                if (blockIdx.x == 0 && s.count > a.max_q_len) raise_device_error(a.c.err, W4A16_ERR_BAD_OFFSETS);
            }
            int64_t upto = n;  // inclusive sum over the threads
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += v;
            }
            __syncthreads();
            if (lane == 31) s_sum[warp] = upto;
            __syncthreads();
            upto += before;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) upto += s_sum[w];
                before += s_sum[w];
            }
            if (round == 0 && a.c.batch <= kThreads) {
                share_out(before, run, runs, shares, run_begin, run_end);
                round = 1;
            }
            if (round == 1 && run_begin >= upto - n && run_begin < upto) {
                s_found[0] = b0 + tid;
                s_found[1] = (int)(run_begin - (upto - n));
            }
            if (round == 1 && before > run_begin) break;
        }
        if (round == 0) share_out(before, run, runs, shares, run_begin, run_end);
        if (run_begin >= run_end) return;
    }
    __syncthreads();

    Cursor at;  // of the computation
    at.b = s_found[0];
    load_sequence(a, at.b, row0, max_rows, at.s);
    at.g = s_found[1] / at.s.blocks;
    at.block = at.s.block + s_found[1] % at.s.blocks;
    at.end = at.s.block + at.s.blocks;
    Cursor to = at;  // of the loads, which run ahead
    int64_t to_load = run_end - run_begin;
    int64_t unit = run_begin;

    // ------------------------------------------------------------- loads --
    unsigned char* ring = smem + warp * kRingBytes;
    const uint32_t ring_u = ptx::smem_u32(ring);
    int pages_from = -1;  // this lane holds the page of block pages_from + lane of the sequence
    int my_page = -1;
    int pages_b = -1;
    // The step of a 16-bit cache.
    auto load_step16 = [&](int stage) {
        if (to_load > 0) {
            if (pages_b != to.b || to.block < pages_from || to.block >= pages_from + 32) {
                pages_b = to.b;
                pages_from = to.block;
                const int p = (to.block + lane) * kBlock + warp * kStep;
                my_page = -1;
                if (p < to.s.length && p + kStep > to.s.low) my_page = (int)page_of(a.c, to.b, p);
            }
            const int page = __shfl_sync(0xffffffffu, my_page, to.block - pages_from);
            const int p0 = to.block * kBlock + warp * kStep;
            const int64_t base = (int64_t)page * a.c.page_stride +
                                 (int64_t)a.c.by_page.remainder(p0) * a.c.slot_stride +
                                 (int64_t)to.g * a.c.head_stride;
            const uint32_t dst = ring_u + stage * L::kStage;
            constexpr int kRowsPer = 32 / L::kChunks;  // rows per instruction
            const int chunk = lane % L::kChunks;
#pragma unroll
            for (int i = 0; i < kStep / kRowsPer; ++i) {
                const int row = i * kRowsPer + lane / L::kChunks;
                const int p = p0 + row;
                // places outside the sequence or before every row's window: zeros, nothing read
                const uint32_t size = page >= 0 && p >= to.s.low && p < to.s.length ? 16u : 0u;
                const int64_t off = size ? base + row * a.c.slot_stride + chunk * 8 : 0;
                ptx::cp_async_16(dst + L::at(row, chunk), a.c.k + off, size);
                ptx::cp_async_16(dst + L::kHalfStage + L::at(row, chunk), a.c.v + off, size);
            }
            --to_load;
            if (++to.block == to.end && to_load > 0) next_item(a, row0, max_rows, turns, to);
        }
        cp_async_commit();
    };

    // Of an 8-bit cache: steps are half as long, so what they cost beside the copies counts. Where a block's rows are
    // is worked out 32 blocks at a time, a lane each.
    int64_t my_rows = -1, my_scales = -1;  // of the lane's block: offsets of the warp's first row and scale in a head
    auto load_step8 = [&](int stage) {
        if (to_load > 0) {
            if (pages_b != to.b || to.block < pages_from || to.block >= pages_from + 32) {
                pages_b = to.b;
                pages_from = to.block;
                const int p = (to.block + lane) * kBlock + warp * kStep;
                my_rows = my_scales = -1;
                if (p < to.s.length && p + kStep > to.s.low) {
                    const int64_t page = page_of(a.c, to.b, p);
                    if (page >= 0) {
                        my_rows = page * a.c.page_stride + (int64_t)a.c.by_page.remainder(p) * a.c.slot_stride;
                        my_scales = page * arg.s.page_stride + a.c.by_page.remainder(p);
                    }
                }
            }
            const int64_t rows = __shfl_sync(0xffffffffu, my_rows, to.block - pages_from);
            const int64_t scales = __shfl_sync(0xffffffffu, my_scales, to.block - pages_from);
            const int p0 = to.block * kBlock + warp * kStep;
            const uint32_t dst = ring_u + stage * L::kStage;
            constexpr int kRowsPer = 32 / L::kChunks;
            const int chunk = lane % L::kChunks, first_row = lane / L::kChunks;
            const uint8_t *k8 = reinterpret_cast<const uint8_t*>(a.c.k), *v8 = reinterpret_cast<const uint8_t*>(a.c.v);
            const int g = head_of(to.g);
            const int64_t first = rows + (int64_t)g * a.c.head_stride + first_row * a.c.slot_stride + chunk * 16;
            const int64_t stride = kRowsPer * a.c.slot_stride;
            const uint8_t *k_row = k8 + first, *v_row = v8 + first;
            if (rows >= 0 && p0 >= to.s.low && p0 + kStep <= to.s.length) {
#pragma unroll
                for (int i = 0; i < kStep / kRowsPer; ++i) {
                    const uint32_t at = dst + L::at(i * kRowsPer + first_row, chunk);
                    ptx::cp_async_16(at, k_row, 16u);
                    ptx::cp_async_16(at + L::kHalfStage, v_row, 16u);
                    k_row += stride;
                    v_row += stride;
                }
            } else {
                // places outside the sequence or before every row's window: zeros, nothing read
#pragma unroll
                for (int i = 0; i < kStep / kRowsPer; ++i) {
                    const int row = i * kRowsPer + first_row;
                    const bool real = rows >= 0 && p0 + row >= to.s.low && p0 + row < to.s.length;
                    const uint32_t at = dst + L::at(row, chunk);
                    ptx::cp_async_16(at, real ? k_row : k8, real ? 16u : 0u);
                    ptx::cp_async_16(at + L::kHalfStage, real ? v_row : v8, real ? 16u : 0u);
                    k_row += stride;
                    v_row += stride;
                }
            }
            // scales of 4 places a lane, keys' and then values'; those of places that are not read, 0
            if (lane < kStep / 2) {
                const int p = p0 + (lane & 3) * 4;
                const bool any = rows >= 0 && p + 4 > to.s.low && p < to.s.length;
                const int64_t at = any ? scales + (int64_t)g * arg.s.head_stride + (lane & 3) * 4 : 0;
                ptx::cp_async_16(dst + 2 * L::kHalfStage + lane * 16, (lane < 4 ? arg.s.k : arg.s.v) + at,
                                 any ? 16u : 0u);
            }
            --to_load;
            if (++to.block == to.end && to_load > 0) next_item(a, row0, max_rows, turns, to);
        }
        cp_async_commit();
    };
    auto load_step = [&](int stage) {
        if constexpr (kHeld8) load_step8(stage);
        else load_step16(stage);
    };

    // ------------------------------------------------------- computation --
    uint32_t qf[kKs][NT][2];
    float o[kKs][NT][4];
    float m[NT][2], l[NT][2];
    float scale[NT][2];  // of the columns' scores (8-bit cache)
    int low[NT][2], high[NT][2];  // places that this lane's columns (rows of q) see
    int all_low = 0, all_high = 0;  // and those that all columns do (8-bit cache)

    auto start_item = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = row0 + n * 8 + grp;
            const bool real = r < at.s.count * ratio;
            const int64_t t = at.s.first + a.by_ratio.quotient(r);
            const uint16_t* q =
                a.q + t * a.q_row_stride + (int64_t)(head_of(at.g) * ratio + a.by_ratio.remainder(r)) * a.q_head_stride;
            if constexpr (kHeld8) {
                // Lane quad holds elements quad * D / 4 + 4 ks to + 3, of keys too: the order of a sum does not matter.
#pragma unroll
                for (int ks = 0; ks < kKs; ++ks) {
                    const uint2 u = real ? __ldg(reinterpret_cast<const uint2*>(q + quad * (D / 4) + ks * 4))
                                         : make_uint2(0u, 0u);
                    qf[ks][n][0] = u.x;
                    qf[ks][n][1] = u.y;
                }
                float up = 1.0f;
                if constexpr (E::kDtype == W4A16_DTYPE_BF16) up = to_fp16_row(qf, n);
#pragma unroll
                for (int j = 0; j < 2; ++j)  // column quad * 2 + j is held by the lanes of that group
                    scale[n][j] = a.scale_log2 * __shfl_sync(0xffffffffu, up, (quad * 2 + j) * 4);
            } else {
#pragma unroll
                for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        qf[ks][n][j] =
                            real ? __ldg(reinterpret_cast<const uint32_t*>(q + ks * 16 + j * 8 + quad * 2)) : 0u;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = row0 + n * 8 + quad * 2 + j;
                const int place = at.s.length - at.s.count + a.by_ratio.quotient(row);
                low[n][j] = first_seen(a, place);
                high[n][j] = row < at.s.count * ratio ? (a.causal ? min(at.s.length, place + 1) : at.s.length) : 0;
                m[n][j] = -INFINITY;
                l[n][j] = 0.0f;
            }
#pragma unroll
            for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[ks][n][i] = 0.0f;
        }
        if constexpr (kHeld8) {
            int lowest = 0, highest = 0x7FFFFFFF;  // (columns that are no rows: anything)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (row0 + n * 8 + quad * 2 + j < at.s.count * ratio) {
                        lowest = max(lowest, low[n][j]);
                        highest = min(highest, high[n][j]);
                    }
            all_low = __reduce_max_sync(0xffffffffu, lowest);
            all_high = __reduce_min_sync(0xffffffffu, highest);
        }
    };

    // `edge`: not all of the places are seen by all columns
    auto compute_step = [&](int stage, auto edge) {
        constexpr bool kEdge = decltype(edge)::value;
        const int p0 = at.block * kBlock + warp * kStep;
        if (p0 >= at.s.length || p0 + kStep <= at.s.low) return;
        const uint32_t kb = ring_u + stage * L::kStage;
        const uint32_t vb = kb + L::kHalfStage;
        float s[2][NT][4];  // two chains of dependent MMAs
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[0][n][i] = s[1][n][i] = 0.0f;
        // The scales of the lane's places, grp and grp + 8.
        [[maybe_unused]] float key_scale[2], value_scale[2], value_log2[2];
        if constexpr (kHeld8) {
            const float* sc = reinterpret_cast<const float*>(ring + stage * L::kStage + 2 * L::kHalfStage);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                key_scale[j] = sc[grp + 8 * j];
                value_scale[j] = sc[kStep + grp + 8 * j];
                value_log2[j] = fmaxf(__log2f(value_scale[j]), kLeastLog2);  // of 0 too, in a cache never appended to
            }
#pragma unroll
            for (int c = 0; c < kKs / 4; ++c) {
                const uint4 x = lds128(kb + L::at(grp, quad * (kKs / 4) + c));
                const uint4 y = lds128(kb + L::at(grp + 8, quad * (kKs / 4) + c));
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t k[4];
                    H::to_fp16(xs[i], k[0], k[2]);
                    H::to_fp16(ys[i], k[1], k[3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma<M>(s[i & 1][n], k, qf[c * 4 + i][n][0], qf[c * 4 + i][n][1]);
                }
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < kKs; ++ks) {
                uint32_t k[4];
                ldmatrix_x4(k, kb + L::at(lane & 15, ks * 2 + (lane >> 4)));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma<M>(s[ks & 1][n], k, qf[ks][n][0], qf[ks][n][1]);
            }
        }
        // With an 8-bit cache the maximum is of s_j + log2(v_j), v_j the value's scale: it is the weights of the
        // second product, 2^(s_j - m) v_j, that have to stay in range. The sum takes 2^(s_j - m), at most 2^96 each.
        bool rise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = p0 + grp + (i >> 1) * 8;
                float v = s[0][n][i] + s[1][n][i];
                if constexpr (kHeld8) v = v * key_scale[i >> 1] * scale[n][i & 1];
                else v *= a.scale_log2;
                if (kEdge && (p < low[n][i & 1] || p >= high[n][i & 1])) v = -INFINITY;
                s[0][n][i] = v;
                if constexpr (kHeld8) s[1][n][i] = kEdge && v == -INFINITY ? v : v + value_log2[i >> 1];
                rise = rise || s[kHeld8][n][i] > m[n][i & 1];
            }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float top = fmaxf(s[kHeld8][n][j], s[kHeld8][n][j + 2]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    top = fmaxf(top, m[n][j]);
                    const float keep = m[n][j] == -INFINITY ? 0.0f : fast_exp2(m[n][j] - top);
                    l[n][j] = rescaled(l[n][j], m[n][j], top);
                    m[n][j] = top;
#pragma unroll
                    for (int ks = 0; ks < kKs; ++ks) {
                        o[ks][n][j] *= keep;
                        o[ks][n][j + 2] *= keep;
                    }
                }
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float base = m[n][i & 1] == -INFINITY ? 0.0f : m[n][i & 1];
                p[i] = fast_exp2(s[0][n][i] - base);
            }
            l[n][0] += p[0] + p[2];
            l[n][1] += p[1] + p[3];
            if constexpr (kHeld8) {
#pragma unroll
                for (int i = 0; i < 4; ++i)  // (a place that is not seen may have any scale; the first product is at most 1)
                    p[i] = kEdge && s[0][n][i] == -INFINITY ? 0.0f : p[i] * value_scale[i >> 1] * kWeightUp;
            }
            pf[n][0] = transpose_8x8(M::pack(p[0], p[1]));
            pf[n][1] = transpose_8x8(M::pack(p[2], p[3]));
        }
        if constexpr (kEdge && H::kFormat == W4A16_CACHE_E4M3) {
            // The bytes of a row whose scale is NaN may be e4m3's NaN, and 0 times that is not 0: they are cleared.
            // The rows that see the place have a weight of NaN.
            bool bad[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) bad[j] = value_scale[j] != value_scale[j];
            if (__any_sync(0xffffffffu, bad[0] || bad[1])) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    for (int c = quad; bad[j] && c < L::kChunks; c += 4)
                        *reinterpret_cast<uint4*>(ring + stage * L::kStage + L::kHalfStage + L::at(grp + 8 * j, c)) =
                            make_uint4(0, 0, 0, 0);
                __syncwarp();
            }
        }
        if constexpr (kHeld8) {
            // Two adjacent elements of a place are one 16-bit unit of the transposing load: bytes 0 and 2 of a
            // register are one element of places 2 quad and 2 quad + 1, bytes 1 and 3 the next. Row grp of tile ks is
            // element 16 ks + 2 grp, row grp + 8 the one after it.
#pragma unroll
            for (int c = 0; c < kKs; c += 2) {
                uint32_t x[4];
                ldmatrix_x4_trans(x, vb + L::at(lane & 15, c + (lane >> 4)));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t v[4];
                    H::to_fp16_apart(x[2 * j], v[0], v[1]);
                    H::to_fp16_apart(x[2 * j + 1], v[2], v[3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma<M>(o[c + j][n], v, pf[n][0], pf[n][1]);
                }
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < kKs; ++ks) {
                uint32_t v[4];
                ldmatrix_x4_trans(v, vb + L::at((lane & 7) + ((lane >> 4) << 3), ks * 2 + ((lane >> 3) & 1)));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma<M>(o[ks][n], v, pf[n][0], pf[n][1]);
            }
        }
    };

    // Adds up the warps' parts of the item that ends here (or whose run ends
    // here) and writes the result, or the part for the last of its thread blocks to join.
    float* join = reinterpret_cast<float*>(smem + kWarps * kRingBytes);
    auto write_row = [&](int r, int d, float (&acc)[8], float top, float sum) {
        if (kHeld8 && at.g * lanes + head0 >= a.c.kv_heads) return;  // (a head too many in the last turn)
        const int64_t row = (int64_t)(at.s.first + a.by_ratio.quotient(row0 + r)) * a.heads +
                            head_of(at.g) * ratio + a.by_ratio.remainder(row0 + r);
        const float inv = sum > 0.0f || sum != sum ? (kHeld8 ? 1.0f / kWeightUp : 1.0f) / sum : 0.0f;
        uint4 w;
        w.x = E::pack(acc[0] * inv, acc[1] * inv);
        w.y = E::pack(acc[2] * inv, acc[3] * inv);
        w.z = E::pack(acc[4] * inv, acc[5] * inv);
        w.w = E::pack(acc[6] * inv, acc[7] * inv);
        *reinterpret_cast<uint4*>(a.out + row * D + d) = w;
        if (a.lse && d == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    };
    auto finish_item = [&](int64_t item_begin, int64_t item_end) {
        const int c0 = shares.owner(item_begin, run), c1 = shares.owner(item_end - 1, run);
        const int64_t slot = 2 * (int64_t)blockIdx.x + (c0 == (int)run ? 1 : 0);
        int* counter = arg.counters + c0 * side + member;
        const int rows = min(at.s.count * ratio - row0, kRows);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], d);
                if (grp == 0) s_stats[warp][n * 8 + quad * 2 + j] = make_float2(m[n][j], l[n][j]);
            }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = quad * 2 + j;
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_stats[w][n * 8 + col].x);
                const float keep = m[n][j] == -INFINITY ? 0.0f : fast_exp2(m[n][j] - top);
#pragma unroll
                for (int ks = 0; ks < kKs; ++ks) {
                    const int d = ks * 16 + (kHeld8 ? 2 * grp : grp);
                    join[L::join_at(warp, col, d)] = o[ks][n][j] * keep;
                    join[L::join_at(warp, col, d + (kHeld8 ? 1 : 8))] = o[ks][n][j + 2] * keep;
                }
            }
            __syncthreads();
            if (tid < 8 * kOutChunks) {
                const int col = tid / kOutChunks, d = tid % kOutChunks * 8;
                const int r = n * 8 + col;
                float top = -INFINITY, sum = 0.0f, acc[8];
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_stats[w][r].x);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 st = s_stats[w][r];
                    sum += rescaled(st.y, st.x, top);
                    const float4* src = reinterpret_cast<const float4*>(join + L::join_at(w, col, d));
                    const float4 x = src[0], y = src[1];
                    acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
                    acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
                }
                if (r < rows) {
                    if (c0 == c1) {
                        write_row(r, d, acc, top, sum);
                    } else {
                        float4* dst = reinterpret_cast<float4*>(arg.parts + (slot * kRows + r) * D + d);
                        __stcg(dst, make_float4(acc[0], acc[1], acc[2], acc[3]));
                        __stcg(dst + 1, make_float4(acc[4], acc[5], acc[6], acc[7]));
                        if (d == 0) __stcg(arg.stats + slot * kRows + r, make_float2(top, sum));
                    }
                }
            }
            if (n + 1 < NT) __syncthreads();
        }
        if (c0 == c1) {
            __syncthreads();  // the shared arrays are free again
            return;
        }
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            const int done = ptx::atom_add_acq_rel_gpu(counter, 1);
            s_last = done == c1 - c0;
            if (s_last) *counter = 0;
        }
        __syncthreads();
        if (!s_last) return;
        __threadfence();
        // a thread per 8 elements of a row; the parts' statistics by way of shared memory, 64 parts at a time
        float2* stats = reinterpret_cast<float2*>(join);  // [64][rows]
        static_assert(64 * kRows * sizeof(float2) <= L::kJoinBytes, "statistics of 64 parts");
        for (int i0 = 0; i0 < rows * kOutChunks; i0 += kThreads) {
            const int i = i0 + tid;
            const bool mine = i < rows * kOutChunks;
            const int r = mine ? i / kOutChunks : 0, d = i % kOutChunks * 8;
            float top = -INFINITY, sum = 0.0f, acc[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
            for (int p0 = c0; p0 <= c1; p0 += 64) {
                const int n = min(64, c1 + 1 - p0);
                auto slot_of = [&](int k) {
                    return (int64_t)(2 * ((p0 + k) * side + member) + (p0 + k == c0));
                };
                __syncthreads();
                for (int k = tid; k < n * rows; k += kThreads) {
                    const int part = k / rows, row = k - part * rows;
                    stats[part * kRows + row] = __ldcg(arg.stats + slot_of(part) * kRows + row);
                }
                __syncthreads();
                if (!mine) continue;
                float higher = top;
                for (int k = 0; k < n; ++k) higher = fmaxf(higher, stats[k * kRows + r].x);
                const float keep = top == -INFINITY ? 0.0f : fast_exp2(top - higher);
                sum = rescaled(sum, top, higher);
                top = higher;
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] *= keep;
#pragma unroll 8
                for (int k = 0; k < n; ++k) {
                    const float4* src = reinterpret_cast<const float4*>(arg.parts + (slot_of(k) * kRows + r) * D + d);
                    const float4 x = __ldcg(src), y = __ldcg(src + 1);
                    const float2 st = stats[k * kRows + r];
                    const float f = st.x == -INFINITY ? 0.0f : fast_exp2(st.x - top);
                    sum += rescaled(st.y, st.x, top);
                    acc[0] += x.x * f; acc[1] += x.y * f; acc[2] += x.z * f; acc[3] += x.w * f;
                    acc[4] += y.x * f; acc[5] += y.y * f; acc[6] += y.z * f; acc[7] += y.w * f;
                }
            }
            if (mine) write_row(r, d, acc, top, sum);
        }
        __syncthreads();  // the shared arrays are free again
    };

    // -------------------------------------------------------------- the run --
    int stage = 0;
#pragma unroll
    for (int i = 0; i < L::kStages - 1; ++i) load_step(i);
    while (true) {
        // the item's blocks in the work list
        const int64_t item_begin = unit - (at.block - at.s.block), item_end = item_begin + at.s.blocks;
        const int64_t stop = min(item_end, run_end);
        start_item();
        for (; unit < stop; ++unit, ++at.block) {
            cp_async_wait<L::kStages - 2>();
            __syncwarp();
            load_step(stage == 0 ? L::kStages - 1 : stage - 1);
            if constexpr (kHeld8) {
                const int p0 = at.block * kBlock + warp * kStep;
                if (p0 >= all_low && p0 + kStep <= all_high) compute_step(stage, std::false_type{});
                else compute_step(stage, std::true_type{});
            } else {
                compute_step(stage, std::true_type{});
            }
            stage = stage + 1 == L::kStages ? 0 : stage + 1;
        }
        finish_item(item_begin, item_end);
        if (unit == run_end) break;
        next_item(a, row0, max_rows, turns, at);
    }
}

// ------------------------------------------------------------------- host --

inline int step_blocks(const DeviceInfo& dev) { return dev.sms * kBlocksPerSm; }

template <class E, class H, int D, int NT>
w4a16_status launch(const DeviceInfo& dev, StepArgs arg, cudaStream_t st) {
    using L = Layout<H, D>;
    const int blocks = step_blocks(dev);
    if constexpr (L::kHeld8) {
        // As many heads side by side as there are, or in as few turns as leave at most 1 thread block in 32 idle.
        const int heads = arg.a.c.kv_heads;
        double best = 0.0;
        for (int turns = 1; turns <= heads && best < 0.97; ++turns) {
            const int lanes = (heads + turns - 1) / turns;
            const double busy = (double)(blocks / (lanes * arg.row_groups)) * arg.row_groups * heads / turns / blocks;
            if (busy <= best) continue;
            best = busy;
            arg.lanes = lanes;
            arg.turns = turns;
        }
    }
    static PerDeviceOnce once;
    const cudaError_t e = once.run(dev.device, [] {
        return cudaFuncSetAttribute(step_kernel<E, H, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    L::kSmem);
    });
    if (e != cudaSuccess) return cuda_status(e, "paged_attention: cudaFuncSetAttribute");
    return launch_overlapped("paged_attention", step_kernel<E, H, D, NT>, dim3((unsigned)blocks), kThreads,
                             L::kSmem, st, arg);
}

// The arguments, with the workspace laid out.
inline StepArgs step_args(const DeviceInfo& dev, const AttentionArgs& a, const ScaleArgs& s, void* workspace) {
    const int blocks = step_blocks(dev);
    StepArgs arg{};
    arg.a = a;
    arg.s = s;
    unsigned char* w = static_cast<unsigned char*>(workspace);
    arg.counters = reinterpret_cast<int*>(w);
    w += align_up((size_t)blocks * sizeof(int));
    arg.stats = reinterpret_cast<float2*>(w);
    w += align_up(2 * (size_t)blocks * kStepRows * sizeof(float2));
    arg.parts = reinterpret_cast<float*>(w);
    return arg;
}

template <class E, class H>
w4a16_status launch_rows(const DeviceInfo& dev, const AttentionArgs& a, const ScaleArgs& s, int max_rows,
                         void* workspace, cudaStream_t st) {
    StepArgs arg = step_args(dev, a, s, workspace);
    const bool two = max_rows > 8;
    arg.row_groups = (max_rows + kStepRows - 1) / kStepRows;
    if (a.c.head_dim == 128)
        return two ? launch<E, H, 128, 2>(dev, arg, st) : launch<E, H, 128, 1>(dev, arg, st);
    return two ? launch<E, H, 64, 2>(dev, arg, st) : launch<E, H, 64, 1>(dev, arg, st);
}

}  // namespace
}  // namespace w4a16
