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
// Measured (heads of 128, 8 cached): one token each of 64 sequences of 300 to
// 8000 places, 1.10 GB: 171 us, 6.4 TB/s, 95% of the copy rate; two of 125000
// and 133000 places, 1.06 GB: 167 us, 6.3 TB/s; one of 777 places 10 us, which is
// latency: 2 us of launch, 1 to find the run, 2 for page entries and then k and
// v, 1 for a block's products with instructions not yet cached, 4 for the join.
#include "attention.cuh"

namespace w4a16 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 16;               // places per warp step
constexpr int kBlock = kWarps * kStep;  // places per block of the work list
constexpr int kBlocksPerSm = 2;
constexpr int kRingBytes = 24 * 1024;   // per warp

template <int D>
struct Layout {
    static constexpr int kRowBytes = D * 2;
    static constexpr int kChunks = D / 8;                       // 16-byte pieces per row
    static constexpr int kHalfStage = kStep * kRowBytes;        // k, then v
    static constexpr int kStages = kRingBytes / (2 * kHalfStage);
    static constexpr int kJoinBytes = kWarps * 8 * D * 4;
    static constexpr int kSmem = kWarps * kRingBytes + kJoinBytes;
    // piece `chunk` of row `row`; eight rows of one chunk fall into eight different bank groups
    __device__ static __forceinline__ uint32_t at(int row, int chunk) {
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

struct StepArgs {
    AttentionArgs a;
    int* counters;   // one per thread block, zero between calls
    float* parts;    // [2 * blocks][rows][D]: o of the parts of divided items
    float2* stats;   // [2 * blocks][rows]: their m and l
};

// A sequence as this kernel sees it; blocks == 0: not one of its own.
struct Sequence {
    int first, count, length;
    int low;         // first place that any row sees
    int block, blocks;  // its 64-place blocks: the first, and how many (one at least, so that empty rows are written)
};

__device__ __forceinline__ void load_sequence(const AttentionArgs& a, int b, int max_rows, Sequence& s) {
    const int first = __ldg(a.c.q_offsets + b), next = __ldg(a.c.q_offsets + b + 1), length = __ldg(a.c.kv_lens + b);
    s.first = first;
    s.count = next - first;
    s.blocks = 0;
    if (first < 0 || next > a.c.T || s.count <= 0 || s.count > a.max_q_len || s.count * a.ratio > max_rows) return;
    s.length = cache_length(a.c, length);
    s.low = first_seen(a, s.length - s.count);
    s.block = s.low / kBlock;
    s.blocks = max(1, (s.length + kBlock - 1) / kBlock - s.block);
}

// This thread block's run of `total` units.
__device__ __forceinline__ void share_out(int64_t total, Shares& shares, int64_t& begin, int64_t& end) {
    shares.base = total / gridDim.x;
    shares.more = (int)(total - shares.base * gridDim.x);
    begin = shares.start(blockIdx.x);
    end = shares.start(blockIdx.x + 1);
}

// A position in the work list, as a warp walks it.
struct Cursor {
    int b, g, block, end;  // block of the sequence, and one past the item's last
    Sequence s;
};

__device__ __forceinline__ void next_item(const AttentionArgs& a, int max_rows, Cursor& c) {
    if (++c.g == a.c.kv_heads) {
        c.g = 0;
        do {
            if (++c.b >= a.c.batch) {  // past the list's end: never used
                c.s.blocks = 0;
                break;
            }
            load_sequence(a, c.b, max_rows, c.s);
        } while (c.s.blocks == 0);
    }
    c.block = c.s.block;
    c.end = c.s.block + c.s.blocks;
}

template <class E, int D, int NT>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) step_kernel(const __grid_constant__ StepArgs arg) {
    using L = Layout<D>;
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

    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (blockIdx.x == 0) check_offsets(a.c);

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
                load_sequence(a, b0 + tid, kRows, s);
                n = (int64_t)s.blocks * a.c.kv_heads;
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
                share_out(before, shares, run_begin, run_end);
                round = 1;
            }
            if (round == 1 && run_begin >= upto - n && run_begin < upto) {
                s_found[0] = b0 + tid;
                s_found[1] = (int)(run_begin - (upto - n));
            }
            if (round == 1 && before > run_begin) break;
        }
        if (round == 0) share_out(before, shares, run_begin, run_end);
        if (run_begin >= run_end) return;
    }
    __syncthreads();

    Cursor at;  // of the computation
    at.b = s_found[0];
    load_sequence(a, at.b, kRows, at.s);
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
    auto load_step = [&](int stage) {
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
            const uint32_t dst = ring_u + stage * 2 * L::kHalfStage;
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
            if (++to.block == to.end && to_load > 0) next_item(a, kRows, to);
        }
        cp_async_commit();
    };

    // ------------------------------------------------------- computation --
    uint32_t qf[kKs][NT][2];
    float o[kKs][NT][4];
    float m[NT][2], l[NT][2];
    int low[NT][2], high[NT][2];  // places that this lane's columns (rows of q) see

    auto start_item = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = n * 8 + grp;
            const bool real = r < at.s.count * ratio;
            const int64_t t = at.s.first + a.by_ratio.quotient(r);
            const uint16_t* q =
                a.q + t * a.q_row_stride + (int64_t)(at.g * ratio + a.by_ratio.remainder(r)) * a.q_head_stride;
#pragma unroll
            for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    qf[ks][n][j] = real ? __ldg(reinterpret_cast<const uint32_t*>(q + ks * 16 + j * 8 + quad * 2)) : 0u;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = n * 8 + quad * 2 + j;
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
    };

    auto compute_step = [&](int stage) {
        const int p0 = at.block * kBlock + warp * kStep;
        if (p0 >= at.s.length || p0 + kStep <= at.s.low) return;
        const uint32_t kb = ring_u + stage * 2 * L::kHalfStage;
        const uint32_t vb = kb + L::kHalfStage;
        float s[2][NT][4];  // two chains of dependent MMAs
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[0][n][i] = s[1][n][i] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < kKs; ++ks) {
            uint32_t k[4];
            ldmatrix_x4(k, kb + L::at(lane & 15, ks * 2 + (lane >> 4)));
#pragma unroll
            for (int n = 0; n < NT; ++n) mma<E>(s[ks & 1][n], k, qf[ks][n][0], qf[ks][n][1]);
        }
        bool rise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = p0 + grp + (i >> 1) * 8;
                float v = (s[0][n][i] + s[1][n][i]) * a.scale_log2;
                if (p < low[n][i & 1] || p >= high[n][i & 1]) v = -INFINITY;
                s[0][n][i] = v;
                rise = rise || v > m[n][i & 1];
            }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float top = fmaxf(s[0][n][j], s[0][n][j + 2]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    top = fmaxf(top, m[n][j]);
                    const float keep = m[n][j] == -INFINITY ? 0.0f : fast_exp2(m[n][j] - top);
                    m[n][j] = top;
                    l[n][j] *= keep;
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
            pf[n][0] = transpose_8x8(E::pack(p[0], p[1]));
            pf[n][1] = transpose_8x8(E::pack(p[2], p[3]));
        }
#pragma unroll
        for (int ks = 0; ks < kKs; ++ks) {
            uint32_t v[4];
            ldmatrix_x4_trans(v, vb + L::at((lane & 7) + ((lane >> 4) << 3), ks * 2 + ((lane >> 3) & 1)));
#pragma unroll
            for (int n = 0; n < NT; ++n) mma<E>(o[ks][n], v, pf[n][0], pf[n][1]);
        }
    };

    // Adds up the warps' parts of the item that ends here (or whose run ends
    // here) and writes the result, or the part for the last of its thread blocks to join.
    float* join = reinterpret_cast<float*>(smem + kWarps * kRingBytes);
    auto write_row = [&](int r, int d, float (&acc)[8], float top, float sum) {
        const int64_t row = (int64_t)(at.s.first + a.by_ratio.quotient(r)) * a.heads + at.g * ratio +
                            a.by_ratio.remainder(r);
        const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
        uint4 w;
        w.x = E::pack(acc[0] * inv, acc[1] * inv);
        w.y = E::pack(acc[2] * inv, acc[3] * inv);
        w.z = E::pack(acc[4] * inv, acc[5] * inv);
        w.w = E::pack(acc[6] * inv, acc[7] * inv);
        *reinterpret_cast<uint4*>(a.out + row * D + d) = w;
        if (a.lse && d == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    };
    auto finish_item = [&](int64_t item_begin, int64_t item_end) {
        const int c0 = shares.owner(item_begin, blockIdx.x), c1 = shares.owner(item_end - 1, blockIdx.x);
        const int64_t slot = 2 * (int64_t)blockIdx.x + (c0 == (int)blockIdx.x ? 1 : 0);
        const int rows = at.s.count * ratio;
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
                    join[L::join_at(warp, col, ks * 16 + grp)] = o[ks][n][j] * keep;
                    join[L::join_at(warp, col, ks * 16 + grp + 8)] = o[ks][n][j + 2] * keep;
                }
            }
            __syncthreads();
            if (tid < 8 * L::kChunks) {
                const int col = tid / L::kChunks, d = tid % L::kChunks * 8;
                const int r = n * 8 + col;
                float top = -INFINITY, sum = 0.0f, acc[8];
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_stats[w][r].x);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 st = s_stats[w][r];
                    sum += st.y * (st.x == -INFINITY ? 0.0f : fast_exp2(st.x - top));  // a sum of NaN stays one
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
            const int done = ptx::atom_add_acq_rel_gpu(arg.counters + c0, 1);
            s_last = done == c1 - c0;
            if (s_last) arg.counters[c0] = 0;
        }
        __syncthreads();
        if (!s_last) return;
        __threadfence();
        // a thread per 8 elements of a row; the parts' statistics by way of shared memory, 64 parts at a time
        float2* stats = reinterpret_cast<float2*>(join);  // [64][rows]
        static_assert(64 * kRows * sizeof(float2) <= L::kJoinBytes, "statistics of 64 parts");
        for (int i0 = 0; i0 < rows * L::kChunks; i0 += kThreads) {
            const int i = i0 + tid;
            const bool mine = i < rows * L::kChunks;
            const int r = mine ? i / L::kChunks : 0, d = i % L::kChunks * 8;
            float top = -INFINITY, sum = 0.0f, acc[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
            for (int p0 = c0; p0 <= c1; p0 += 64) {
                const int n = min(64, c1 + 1 - p0);
                auto slot_of = [&](int k) { return (int64_t)(2 * (p0 + k) + (p0 + k == c0)); };
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
                top = higher;
                sum *= keep;
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] *= keep;
#pragma unroll 8
                for (int k = 0; k < n; ++k) {
                    const float4* src = reinterpret_cast<const float4*>(arg.parts + (slot_of(k) * kRows + r) * D + d);
                    const float4 x = __ldcg(src), y = __ldcg(src + 1);
                    const float2 st = stats[k * kRows + r];
                    const float f = st.x == -INFINITY ? 0.0f : fast_exp2(st.x - top);
                    sum += st.y * f;
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
            compute_step(stage);
            stage = stage + 1 == L::kStages ? 0 : stage + 1;
        }
        finish_item(item_begin, item_end);
        if (unit == run_end) break;
        next_item(a, kRows, at);
    }
}

// ------------------------------------------------------------------- host --

template <class E, int D, int NT>
w4a16_status launch(const DeviceInfo& dev, const StepArgs& arg, int blocks, cudaStream_t st) {
    static PerDeviceOnce once;
    const cudaError_t e = once.run(dev.device, [] {
        return cudaFuncSetAttribute(step_kernel<E, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    Layout<D>::kSmem);
    });
    if (e != cudaSuccess) return cuda_status(e, "paged_attention: cudaFuncSetAttribute");
    return launch_overlapped("paged_attention", step_kernel<E, D, NT>, dim3((unsigned)blocks), kThreads,
                             Layout<D>::kSmem, st, arg);
}

int step_blocks(const DeviceInfo& dev) { return dev.sms * kBlocksPerSm; }

}  // namespace

size_t attention_step_workspace_bytes(const DeviceInfo& dev, int head_dim) {
    const size_t n = (size_t)step_blocks(dev);
    return align_up(n * sizeof(int)) + align_up(2 * n * kStepRows * sizeof(float2)) +
           2 * n * kStepRows * head_dim * sizeof(float);
}

w4a16_status attention_step_launch(const DeviceInfo& dev, int dtype, const AttentionArgs& a, int max_rows,
                                   void* workspace, cudaStream_t st) {
    const int blocks = step_blocks(dev);
    StepArgs arg{};
    arg.a = a;
    unsigned char* w = static_cast<unsigned char*>(workspace);
    arg.counters = reinterpret_cast<int*>(w);
    w += align_up((size_t)blocks * sizeof(int));
    arg.stats = reinterpret_cast<float2*>(w);
    w += align_up(2 * (size_t)blocks * kStepRows * sizeof(float2));
    arg.parts = reinterpret_cast<float*>(w);
    const bool f16 = dtype == W4A16_DTYPE_F16, wide = a.c.head_dim == 128, two = max_rows > 8;
#define W4A16_STEP(D, NT) \
    return f16 ? launch<Fp16, D, NT>(dev, arg, blocks, st) : launch<Bf16, D, NT>(dev, arg, blocks, st)
    if (wide && two) W4A16_STEP(128, 2);
    if (wide) W4A16_STEP(128, 1);
    if (two) W4A16_STEP(64, 2);
    W4A16_STEP(64, 1);
#undef W4A16_STEP
}

}  // namespace w4a16
