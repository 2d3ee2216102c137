// Attention over the paged cache for many rows (chunks of new tokens): tiles of
// 256 rows, a row being one query head of one new token and the rows of a tile
// sharing one cached head, against blocks of 128 places on the tensor cores
// (sm_103a: TMA, tcgen05 MMA, TMEM).
//
// One pass over the places with the running maximum m and sum l of the
// softmax: p = 2^(c s - m), l += sum p, o = o 2^(m - m') + p v whenever m moves
// to m', which it only does when a score passes it by more than 8 (so p stays
// below 2^8 and the read-scale-write of o is rare; out = o / l whatever m is).
//
// 4 D operations per (row, place) bound it: per block of 128 places and
// half tile of 128 rows two 128 x 128 x D products, 512 cycles each at D = 128,
// against 128 exponentials per row. The two halves of a tile take turns: while
// one half's scores go through the softmax, the tensor core forms the other's
// products, and each k and v block that is read serves 256 rows.
//
//   warps 0-3, 4-7  softmax of the two halves: thread = row = TMEM lane. Reads
//                   its 128 scores (tcgen05.ld), writes p as 16-bit pairs over
//                   the first half of the same columns, where the second
//                   product takes it as its A operand. Also fetches its half's
//                   queries (rows of different tokens and heads: cp.async into the
//                   swizzled layout) while the last block of the tile before
//                   it is in work, and writes the result.
//   warp 8          TMA: k and v blocks into a ring of shared memory, one box per page piece and
//                   64 elements. Pages that hold nothing to see are not read:
//                   a box outside the cache reads as zeros.
//   warp 9          MMA issue (warps 10 and 11 only fill the warpgroup): p v of block j, then q k of block j + 1, for one half
//                   and then the other. Slots past a sequence's last place are zeroed in
//                   the v block first (0 times whatever they hold might not be 0).
//
// TMEM: scores (and p) of the halves in columns [0, 128) and [128, 256), o in
// [256, 256 + D) and [256 + D, 256 + 2 D).
//
// The work list (sequence, tile, cached head, block) is cut into equal runs,
// one per SM, on the device; tiles that a cut divides are joined through the
// workspace as in attention_step.cu.
//
// Every mbarrier wait is bounded in time; one that gives up records
// W4A16_ERR_TIMEOUT and the thread block unwinds (its copies and MMAs finish, TMEM is freed).
#include <cudaTypedefs.h>

#include <mutex>

#include "attention.cuh"

namespace w4a16 {
namespace {

constexpr int kHalf = 128;       // rows of a half tile: MMA M, TMEM lanes
constexpr int kTile = 2 * kHalf;
constexpr int kBlock = 128;      // places per block: MMA N of the scores, K of the output
constexpr int kThreads = 384;
// Registers: a launch of 384 threads has 168 each; the two softmax warpgroups
// hold a row of 128 scores a thread and take 216, the third keeps 72 (2 * 216 + 72 = 3 * 168).
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOutCol = 256;
constexpr float kSlack = 8.0f;   // how far a score may pass the running maximum (log2)
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 1000000000ull;

#ifdef W4A16_TEST_HOOKS
__device__ TestHooks g_hooks = {kWaitLimitNs, -1};
__device__ TestCounters g_counters = {0ull, 0ull};
__device__ __forceinline__ uint64_t wait_limit() { return g_hooks.wait_limit_ns; }
__device__ __forceinline__ bool may_issue(int issued) { return g_hooks.issue_limit < 0 || issued < g_hooks.issue_limit; }
#define W4A16_COUNT_TMEM(field) atomicAdd(&g_counters.field, 1ull)
#else
__device__ __forceinline__ constexpr uint64_t wait_limit() { return kWaitLimitNs; }
__device__ __forceinline__ constexpr bool may_issue(int) { return true; }
#define W4A16_COUNT_TMEM(field) ((void)0)
#endif

template <int D>
struct Layout {
    static constexpr int kSlabs = D / 64;              // 64-element slabs: 128-byte swizzled rows
    static constexpr int kSlabBytes = kBlock * 128;
    static constexpr int kStageBytes = kSlabs * kSlabBytes;  // one k or v block; also half a tile's queries
    static constexpr int kStages = (224 * 1024 - 2 * kStageBytes) / kStageBytes;
    static constexpr int kRingAt = 2 * kStageBytes;
    static constexpr int kBarsAt = kRingAt + kStages * kStageBytes;
    static constexpr int kSmem = kBarsAt + 1024 + 1024;  // barriers, and the 1024-byte alignment
};

constexpr int kMaxStages = 12;

struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages];  // ring
    uint64_t q_full[2];   // a half's queries are in shared memory
    uint64_t s_full[2];   // a half's scores are in TMEM (and its o is up to date)
    uint64_t p_full[2];   // a half's p is in TMEM
    uint64_t o_done[2];   // a half's o is complete for the tile
    uint64_t part_in[2];  // a half's threads have written their part
    uint64_t part_out[2]; // whether it was the last of its tile is known
    uint64_t mma_done;
    uint32_t tmem;
    int abort;
    int last[2];
};
static_assert(sizeof(Bars) <= 1024, "barriers");

struct TileArgs {
    AttentionArgs a;
    int* counters;  // two per thread block, zero between calls
    float* parts;   // [2 * blocks][D][256]: o of the parts of divided tiles
    float2* stats;  // [2 * blocks][256]: their m and l
    int min_rows;   // sequences with fewer rows per cached head are attention_step.cu's
    int box;        // places per TMA box
};

struct Sequence {
    int first, count, length;
    int tiles;  // 0: not one of this kernel's
};

__device__ __forceinline__ void load_sequence(const TileArgs& x, int b, Sequence& s) {
    const AttentionArgs& a = x.a;
    s.first = __ldg(a.c.q_offsets + b);
    s.count = __ldg(a.c.q_offsets + b + 1) - s.first;
    s.tiles = 0;
    const int ratio = a.heads / a.c.kv_heads;
    if (s.count <= 0 || s.count > a.max_q_len || (int64_t)s.count * ratio < x.min_rows || s.first < 0 ||
        (int64_t)s.first + s.count > a.c.T)
        return;
    s.length = cache_length(a.c, b);
    s.tiles = (int)(((int64_t)s.count * ratio + kTile - 1) / kTile);
}

// The places that rows [r0, r1) of a sequence see together, and their blocks.
struct Range {
    int low, block, end;  // block == end: none
};

__device__ __forceinline__ Range range_of(const AttentionArgs& a, int count, int length, int64_t r0, int64_t r1) {
    const int ratio = a.heads / a.c.kv_heads;
    const int64_t rows = (int64_t)count * ratio;
    if (r1 > rows) r1 = rows;
    Range r{0, 0, 0};
    if (r0 >= r1) return r;
    const int first = length - count + (int)(r0 / ratio), last = length - count + (int)((r1 - 1) / ratio);
    const int high = a.causal ? min(length, last + 1) : length;
    if (high <= 0) return r;
    r.low = a.window > 0 ? max(0, first - a.window + 1) : 0;
    r.block = r.low / kBlock;
    r.end = (high + kBlock - 1) / kBlock;
    return r;
}

// A tile, and the stretch of its blocks that a thread block computes.
struct Segment {
    int b, tile, g;
    Sequence s;
    Range half0, half1;   // all that the halves see
    int low, block, end;  // of the whole tile; end > block even if nothing is seen
    int from, to;         // the stretch
    __device__ __forceinline__ int begin_of(int w) const { return max(w ? half1.block : half0.block, from); }
    __device__ __forceinline__ int end_of(int w) const { return min(w ? half1.end : half0.end, to); }
    __device__ __forceinline__ bool active(int w, int j) const { return j >= begin_of(w) && j < end_of(w); }
    __device__ __forceinline__ int count_of(int w) const { return max(0, end_of(w) - begin_of(w)); }
};

__device__ __forceinline__ void set_tile(const AttentionArgs& a, Segment& s) {
    const int64_t r = (int64_t)s.tile * kTile;
    s.half0 = range_of(a, s.s.count, s.s.length, r, r + kHalf);
    s.half1 = range_of(a, s.s.count, s.s.length, r + kHalf, r + kTile);
    const bool first = s.half0.end > s.half0.block, second = s.half1.end > s.half1.block;
    s.low = first ? s.half0.low : s.half1.low;
    s.block = first ? s.half0.block : s.half1.block;
    s.end = max(s.half0.end, s.half1.end);
    if (!first && !second) {
        s.block = 0;
        s.end = 1;
    }
}

__device__ __forceinline__ void next_segment(const TileArgs& x, int64_t left, Segment& s) {
    if (++s.g == x.a.c.kv_heads) {
        s.g = 0;
        if (++s.tile == s.s.tiles) {
            s.tile = 0;
            do {
                if (++s.b >= x.a.c.batch) return;  // past the list's end: not reached while units are left
                load_sequence(x, s.b, s.s);
            } while (s.s.tiles == 0);
        }
        set_tile(x.a, s);
    }
    s.from = s.block;
    s.to = (int)min((int64_t)s.end, s.block + left);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(ptx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(ptx::smem_u32(bar))
        : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// v block as the B operand of p v: 64-element slabs of 128-byte rows, a row per
// place (the contraction), so N is contiguous: slabs kSlabBytes apart, 8-place groups 1024 bytes.
__device__ __forceinline__ uint64_t desc_v(uint32_t addr, int slab_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(slab_bytes >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

template <class E>
__host__ __device__ constexpr uint32_t idesc(int n, bool b_n_major) {
    const uint32_t type = E::kDtype == W4A16_DTYPE_BF16 ? 1u : 0u;
    return ptx::idesc_f16_f32(kHalf, n) | (type << 7) | (type << 10) | ((b_n_major ? 1u : 0u) << 16);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// (a.x * s + t, a.y * s + t) in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 s, float2 t) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&s)),
          "l"(*reinterpret_cast<uint64_t*>(&t)));
    return *reinterpret_cast<float2*>(&d);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
    return *reinterpret_cast<float2*>(&d);
}

__device__ __forceinline__ void fail(const TileArgs& x, Bars* bars) {
    *(volatile int*)&bars->abort = 1;
    raise_device_error(x.a.c.err, W4A16_ERR_TIMEOUT);
}

// The list's length, and where this thread block's run starts in it. All
// threads; scratch: 5 * kThreads ints of shared memory. Returns false where there is no run.
struct Run {
    Shares shares;
    int64_t begin, end;
};

__device__ bool find_run(const TileArgs& x, int* scratch, Run& run, Segment& at) {
    __shared__ int64_t s_sum[kThreads / 32];
    __shared__ int64_t s_found[3];
    int* s_first = scratch;  // first tile of each sequence of this round
    int* s_count = scratch + kThreads + 1;
    int* s_length = s_count + kThreads;
    const AttentionArgs& a = x.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto scan = [&](int64_t v, int64_t& all) {  // inclusive, over the threads
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += u;
        }
        __syncthreads();
        if (lane == 31) s_sum[warp] = v;
        __syncthreads();
        all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) v += s_sum[w];
            all += s_sum[w];
        }
        return v;
    };
    int64_t total = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int64_t before = 0;
        for (int b0 = 0; b0 < a.c.batch; b0 += kThreads) {
            Sequence s;
            s.tiles = 0;
            if (b0 + tid < a.c.batch) {
                load_sequence(x, b0 + tid, s);
                if (blockIdx.x == 0 && pass == 0 && s.count > a.max_q_len)
                    raise_device_error(a.c.err, W4A16_ERR_BAD_OFFSETS);
            }
            int64_t tiles;
            const int64_t upto = scan(s.tiles, tiles);  // T rows at most: tiles fit an int
            s_first[tid] = (int)(upto - s.tiles);
            s_count[tid] = s.count;
            s_length[tid] = s.length;
            __syncthreads();
            for (int64_t i0 = 0; i0 < tiles; i0 += kThreads) {
                const int64_t i = i0 + tid;
                int64_t n = 0;
                int lo = 0;
                if (i < tiles) {
                    int hi = kThreads - 1;  // the last sequence that starts at or before tile i
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) >> 1;
                        if (s_first[mid] <= i) lo = mid;
                        else hi = mid - 1;
                    }
                    Segment t;
                    t.tile = (int)(i - s_first[lo]);
                    t.s.count = s_count[lo];
                    t.s.length = s_length[lo];
                    set_tile(a, t);
                    n = (int64_t)(t.end - t.block) * a.c.kv_heads;
                }
                int64_t all;
                const int64_t sum = before + scan(n, all);
                before += all;
                if (pass == 1 && n > 0 && run.begin >= sum - n && run.begin < sum) {
                    s_found[0] = b0 + lo;
                    s_found[1] = i - s_first[lo];
                    s_found[2] = run.begin - (sum - n);
                }
            }
            __syncthreads();
            if (pass == 1 && before > run.begin) break;
        }
        if (pass == 0) {
            total = before;
            run.shares.base = total / gridDim.x;
            run.shares.more = total % gridDim.x;
            run.begin = run.shares.start(blockIdx.x);
            run.end = run.shares.start(blockIdx.x + 1);
            if (run.begin >= run.end) return false;
        }
    }
    at.b = (int)s_found[0];
    at.tile = (int)s_found[1];
    load_sequence(x, at.b, at.s);
    set_tile(a, at);
    at.g = (int)(s_found[2] / (at.end - at.block));
    at.from = at.block + (int)(s_found[2] % (at.end - at.block));
    at.to = (int)min((int64_t)at.end, at.from + (run.end - run.begin));
    return true;
}

template <class E, int D>
__global__ void __launch_bounds__(kThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                const __grid_constant__ TileArgs x) {
    using L = Layout<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* ring = smem + L::kRingAt;
    Bars* bars = reinterpret_cast<Bars*>(smem + L::kBarsAt);
    const AttentionArgs& a = x.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ratio = a.heads / a.c.kv_heads;

    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (blockIdx.x == 0) check_offsets(a.c);
    Run run;
    Segment seg;
    if (!find_run(x, reinterpret_cast<int*>(ring), run, seg)) return;  // the same for all threads
    if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < L::kStages; ++i) {
                ptx::mbar_init(&bars->full[i], 1);
                ptx::mbar_init(&bars->empty[i], 1);
            }
            for (int w = 0; w < 2; ++w) {
                ptx::mbar_init(&bars->q_full[w], kHalf);
                ptx::mbar_init(&bars->s_full[w], 1);
                ptx::mbar_init(&bars->p_full[w], kHalf / 32);
                ptx::mbar_init(&bars->o_done[w], 1);
                ptx::mbar_init(&bars->part_in[w], kHalf);
                ptx::mbar_init(&bars->part_out[w], 1);
            }
            ptx::mbar_init(&bars->mma_done, 1);
            bars->abort = 0;
            ptx::fence_mbar_init();
            ptx::prefetch_tensormap(&map_k);
            ptx::prefetch_tensormap(&map_v);
        }
        __syncwarp();
        ptx::tmem_alloc(&bars->tmem, kTmemCols);
        ptx::tmem_relinquish();
        if (lane == 0) W4A16_COUNT_TMEM(tmem_allocs);
    }
    ptx::fence_proxy_async_shared();  // the scratch above was the ring's memory
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = bars->tmem;
    volatile int* abort = &bars->abort;
    int64_t left = run.end - run.begin;  // units of this run from the segment on
    bool ok = true;

    if (warp >= kLoadWarp) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
      if (warp == kLoadWarp) {
        // ------------------------------------------------------------- loads
        const int pieces = kBlock / x.box;
        const int piece = lane / L::kSlabs, slab = lane % L::kSlabs;
        int issued = 0;
        while (ok) {
            for (int j = seg.from; ok && j < seg.to; ++j) {
                const int p = j * kBlock + piece * x.box;
                int64_t page = a.c.pages;  // outside the cache: zeros
                if (piece < pieces && p < seg.s.length && p + x.box > seg.low) {
                    page = page_of(a.c, seg.b, p);
                    if (page < 0) page = a.c.pages;
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int st = issued % L::kStages, round = issued / L::kStages;
                    ok = may_issue(issued) &&
                         (round == 0 || ptx::mbar_wait(&bars->empty[st], (round - 1) & 1, abort, wait_limit()));
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) ptx::mbar_arrive_expect_tx(&bars->full[st], L::kStageBytes);
                    __syncwarp();
                    if (piece < pieces)
                        tma_load_4d(ring + st * L::kStageBytes + slab * L::kSlabBytes + piece * x.box * 128,
                                    kv ? &map_v : &map_k, &bars->full[st], slab * 64, p % a.c.page_size, seg.g,
                                    (int)page);
                    ++issued;
                }
            }
            left -= seg.to - seg.from;
            if (!ok || left == 0) break;
            next_segment(x, left, seg);
        }
        if (!ok && lane == 0) {
            fail(x, bars);
            volatile int never = 0;  // our own copies land before the thread block ends
            for (int i = max(0, issued - L::kStages); i < issued; ++i)
                ptx::mbar_wait(&bars->full[i % L::kStages], (i / L::kStages) & 1, &never, kDrainLimitNs);
        }
        __syncwarp();
      } else if (warp == kMmaWarp) {
        // --------------------------------------------------------------- MMA
        constexpr uint32_t kIdescS = idesc<E>(kBlock, false), kIdescO = idesc<E>(D, true);
        const uint32_t smem_u = ptx::smem_u32(smem), ring_u = ptx::smem_u32(ring);
        int used = 0;                  // ring stages taken
        int nq[2] = {0, 0}, np[2] = {0, 0};
        auto wait = [&](uint64_t* bar, int n) {  // for its n-th completion, from 0
            if (ok && !ptx::mbar_wait(bar, n & 1, abort, wait_limit())) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            ptx::tc_fence_after();
            return ok;
        };
        auto scores = [&](int w, int st) {
            if (lane == 0) {
                const uint64_t q = ptx::smem_desc_sw128(smem_u + w * L::kStageBytes);
                const uint64_t k = ptx::smem_desc_sw128(ring_u + st * L::kStageBytes);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint64_t at = (uint64_t)(((ks >> 2) * L::kSlabBytes + (ks & 3) * 32) >> 4);
                    mma_ss(tmem + w * kBlock, q + at, k + at, kIdescS, ks > 0);
                }
                ptx::mma_commit(&bars->s_full[w]);
            }
            __syncwarp();
        };
        auto output = [&](int w, int st, bool first, bool last) {
            if (lane == 0) {
                const uint64_t v = desc_v(ring_u + st * L::kStageBytes, L::kSlabBytes);
#pragma unroll
                for (int kk = 0; kk < kBlock / 16; ++kk)
                    ptx::mma_f16_ts(tmem + kOutCol + w * D, tmem + w * kBlock + kk * 8, v + (uint64_t)((kk * 2048) >> 4),
                                    kIdescO, !first || kk > 0);
                if (last) ptx::mma_commit(&bars->o_done[w]);
            }
            __syncwarp();
        };
        // the first block's scores
        int j = seg.from;
        wait(&bars->full[0], 0);
        used = 1;
#pragma unroll
        for (int w = 0; w < 2; ++w)
            if (ok && seg.active(w, j) && wait(&bars->q_full[w], nq[w]++)) scores(w, 0);
        if (lane == 0) ptx::mma_commit(&bars->empty[0]);
        Segment nxt = seg;
        while (ok) {
            // block j of seg, and the block after it: block i of nxt
            int i = j + 1;
            bool more = true;
            const bool turn = i == seg.to;
            if (turn) {
                left -= seg.to - seg.from;
                more = left > 0;
                if (more) {
                    next_segment(x, left, nxt);
                    i = nxt.from;
                }
            }
            const int vst = used % L::kStages, vround = used / L::kStages;
            const int kst = (used + 1) % L::kStages, kround = (used + 1) / L::kStages;
            wait(&bars->full[vst], vround);
            // slots past the last place, in a page that holds it
            const int past = seg.s.length - j * kBlock;
            if (ok && past > 0 && past < kBlock && past % x.box != 0) {
                const int upto = (past + x.box - 1) / x.box * x.box;
                for (int k = lane; k < (upto - past) * (D / 8); k += 32) {
                    const int row = past + k / (D / 8), piece = k % (D / 8);
                    *reinterpret_cast<uint4*>(ring + vst * L::kStageBytes + (piece >> 3) * L::kSlabBytes + row * 128 +
                                              (piece & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                ptx::fence_proxy_async_shared();
                __syncwarp();
            }
            bool k_ready = false;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (ok && seg.active(w, j) && wait(&bars->p_full[w], np[w]++))
                    output(w, vst, j == seg.begin_of(w), j == seg.end_of(w) - 1);
                if (w == 1 && lane == 0) ptx::mma_commit(&bars->empty[vst]);
                if (more && !k_ready) {
                    wait(&bars->full[kst], kround);
                    k_ready = true;
                }
                if (ok && more && nxt.active(w, i) &&
                    (i != nxt.begin_of(w) || wait(&bars->q_full[w], nq[w]++)))
                    scores(w, kst);
            }
            if (more && lane == 0) ptx::mma_commit(&bars->empty[kst]);
            used += 2;
            if (!more) break;
            if (turn) seg = nxt;
            j = i;
        }
        if (lane == 0) {
            if (!ok) fail(x, bars);
            ptx::mma_commit(&bars->mma_done);
            volatile int never = 0;
            ptx::mbar_wait(&bars->mma_done, 0, &never, kDrainLimitNs);
        }
        __syncwarp();
      }
    } else {
        // ----------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int w = warp >> 2;
        const int row = tid & (kHalf - 1);
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_addr = lane_base + w * kBlock, o_addr = lane_base + kOutCol + w * D;
        const uint32_t q_smem = ptx::smem_u32(smem) + w * L::kStageBytes;
        int ns = 0, no = 0, nj = 0;
        // this half's queries of a tile, 16 bytes a lane; rows past the sequence's are zeros
        auto load_q = [&](const Segment& s) {
            constexpr int kPieces = D / 8, kRowsPer = 32 / kPieces;
            const int piece = lane % kPieces;
#pragma unroll 4
            for (int i = 0; i < 32 / kRowsPer; ++i) {
                const int r = (warp & 3) * 32 + i * kRowsPer + lane / kPieces;
                const int64_t at = (int64_t)s.tile * kTile + w * kHalf + r;
                const int64_t token = at / ratio;
                const bool real = token < s.s.count;
                const uint16_t* src = a.q + (real ? (s.s.first + token) * a.q_row_stride +
                                                        (s.g * ratio + at % ratio) * a.q_head_stride + piece * 8
                                                  : 0);
                ptx::cp_async_16(q_smem + (piece >> 3) * L::kSlabBytes + r * 128 + (((piece & 7) ^ (r & 7)) << 4), src,
                                 real ? 16u : 0u);
            }
        };
        auto q_ready = [&] {
            ptx::cp_async_wait_all();
            ptx::fence_proxy_async_shared();
            ptx::mbar_arrive(&bars->q_full[w]);
        };
        if (seg.count_of(w) > 0) {
            load_q(seg);
            q_ready();
        }
        int64_t unit = run.begin;  // of the segment's first block
        while (true) {
            const int begin = seg.begin_of(w), n = seg.count_of(w);
            left -= seg.to - seg.from;
            Segment nxt = seg;
            if (left > 0) next_segment(x, left, nxt);
            const bool load_next = left > 0 && nxt.count_of(w) > 0;
            const int64_t at = (int64_t)seg.tile * kTile + w * kHalf + row;
            const int64_t token = at / ratio;
            const bool real = token < seg.s.count;
            const int place = seg.s.length - seg.s.count + (int)token;
            const int low = a.window > 0 ? max(0, place - a.window + 1) : 0;
            const int high = !real ? 0 : a.causal ? min(seg.s.length, place + 1) : seg.s.length;
            float m = -INFINITY;
            float2 sum = make_float2(0.0f, 0.0f);
            for (int j = begin; j < begin + n; ++j) {
                if (!ptx::mbar_wait(&bars->s_full[w], ns & 1, abort, wait_limit())) ok = false;
                ++ns;
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                if (j == begin + n - 1 && load_next) load_q(nxt);  // the last scores are formed: q may go
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) ptx::tmem_ld_32x32b_x32(s_addr + c * 32, s[c]);
                ptx::tmem_ld_wait();
                const int p0 = j * kBlock;
                if (__any_sync(0xffffffffu, low > p0 || high < p0 + kBlock)) {
                    const int lo = low - p0, hi = high - p0;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c * 32 + i < lo || c * 32 + i >= hi) s[c][i] = 0xFF800000u;  // -infinity
                }
                float top = __uint_as_float(s[0][0]), top2 = __uint_as_float(s[0][1]);
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        top = max3(top, __uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1]));
                        top2 = max3(top2, __uint_as_float(s[c][i + 2]), __uint_as_float(s[c][i + 3]));
                    }
                top = fmaxf(top, top2) * a.scale_log2;
                if (__any_sync(0xffffffffu, top > m + kSlack)) {
                    top = fmaxf(top, m);
                    const float keep = m == -INFINITY ? 0.0f : fast_exp2(m - top);
                    m = top;
                    sum.x *= keep;
                    sum.y *= keep;
                    if (j > begin) {  // p v of the block before is done: these scores were formed after it
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            ptx::tmem_ld_32x32b_x16(o_addr + c, o);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
                            ptx::tmem_st_32x32b_x16(o_addr + c, o);
                        }
                        ptx::tmem_st_wait();
                    }
                }
                const float base = m == -INFINITY ? 0.0f : -m;
                const float2 c2 = make_float2(a.scale_log2, a.scale_log2), m2 = make_float2(base, base);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 e = fma2(make_float2(__uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1])), c2,
                                        m2);
                        e.x = fast_exp2(e.x);
                        e.y = fast_exp2(e.y);
                        sum = add2(sum, e);
                        p[i] = E::pack(e.x, e.y);
                    }
                    ptx::tmem_st_32x32b_x16(s_addr + c * 16, p);
                }
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bars->p_full[w]);
            }
            if (!ok) break;
            if (load_next) {
                if (n == 0) load_q(nxt);
                q_ready();
            }
            // ---- the tile's result, or this thread block's part of it
            if (n > 0) {
                if (!ptx::mbar_wait(&bars->o_done[w], no & 1, abort, wait_limit())) ok = false;
                ++no;
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
            }
            float l = sum.x + sum.y;
            const int64_t item = unit - (seg.from - seg.block);
            const int64_t c0 = run.shares.owner(item), c1 = run.shares.owner(item + (seg.end - seg.block) - 1);
            const int64_t out_row = (seg.s.first + token) * a.heads + seg.g * ratio + at % ratio;
            auto write32 = [&](int d, const float (&v)[32], float scale) {
                uint4* dst = reinterpret_cast<uint4*>(a.out + out_row * D + d);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    dst[i] = make_uint4(E::pack(v[8 * i] * scale, v[8 * i + 1] * scale),
                                        E::pack(v[8 * i + 2] * scale, v[8 * i + 3] * scale),
                                        E::pack(v[8 * i + 4] * scale, v[8 * i + 5] * scale),
                                        E::pack(v[8 * i + 6] * scale, v[8 * i + 7] * scale));
            };
            auto write_lse = [&](float top, float total) {
                if (a.lse) a.lse[out_row] = total == 0.0f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
            };
            const int64_t slot = 2 * (int64_t)blockIdx.x + (c0 == blockIdx.x ? 1 : 0);
            const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
                uint32_t r[32];
                float v[32];
                if (n > 0) {
                    ptx::tmem_ld_32x32b_x32(o_addr + d, r);
                    ptx::tmem_ld_wait();
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = n > 0 ? __uint_as_float(r[i]) : 0.0f;
                if (c0 == c1) {
                    if (real) write32(d, v, inv);
                } else {
                    float* dst = x.parts + (slot * D + d) * kTile + w * kHalf + row;
#pragma unroll
                    for (int i = 0; i < 32; ++i) __stcg(dst + i * kTile, v[i]);
                }
            }
            ptx::tc_fence_before();  // o may be overwritten once the next p is announced
            if (c0 == c1) {
                if (real) write_lse(m, l);
            } else {
                __stcg(x.stats + slot * kTile + w * kHalf + row, make_float2(m, l));
                __threadfence();
                ptx::mbar_arrive(&bars->part_in[w]);
                if (row == 0 && ptx::mbar_wait(&bars->part_in[w], nj & 1, abort, wait_limit())) {
                    const int done = ptx::atom_add_acq_rel_gpu(x.counters + 2 * c0 + w, 1);
                    bars->last[w] = done == (int)(c1 - c0);
                    if (bars->last[w]) x.counters[2 * c0 + w] = 0;
                    ptx::mbar_arrive(&bars->part_out[w]);
                }
                __syncwarp();
                if (!ptx::mbar_wait(&bars->part_out[w], nj & 1, abort, wait_limit())) ok = false;
                ++nj;
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                if (bars->last[w]) {
                    __threadfence();
                    const float2* st = x.stats + w * kHalf + row;
                    float top = -INFINITY, total = 0.0f;
                    for (int64_t c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(st + (2 * c + (c == c0)) * kTile).x);
                    for (int64_t c = c0; c <= c1; ++c) {
                        const float2 v = __ldcg(st + (2 * c + (c == c0)) * kTile);
                        total += v.x == -INFINITY ? 0.0f : v.y * fast_exp2(v.x - top);
                    }
                    const float inv_total = total > 0.0f || total != total ? 1.0f / total : 0.0f;
#pragma unroll 1
                    for (int d = 0; d < D; d += 32) {
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0.0f;
                        for (int64_t c = c0; c <= c1; ++c) {
                            const int64_t part = 2 * c + (c == c0);
                            const float mc = __ldcg(st + part * kTile).x;
                            const float f = mc == -INFINITY ? 0.0f : fast_exp2(mc - top);
                            const float* src = x.parts + (part * D + d) * kTile + w * kHalf + row;
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] += f * __ldcg(src + i * kTile);
                        }
                        if (real) write32(d, v, inv_total);
                    }
                    if (real) write_lse(top, total);
                }
            }
            if (left == 0) break;
            unit += seg.to - seg.from;
            seg = nxt;
        }
        ptx::cp_async_wait_all();
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kMmaWarp) {
        ptx::tmem_dealloc(tmem, kTmemCols);
        if (lane == 0) W4A16_COUNT_TMEM(tmem_frees);
    }
}

// ------------------------------------------------------------------- host --

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

template <class E, int D>
w4a16_status launch(const DeviceInfo& dev, const TileArgs& x, cudaStream_t st) {
    using L = Layout<D>;
    static_assert(L::kStages <= kMaxStages, "ring");
    static PerDeviceOnce once;
    const cudaError_t e = once.run(dev.device, [] {
        return cudaFuncSetAttribute(tile_kernel<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    });
    if (e != cudaSuccess) return cuda_status(e, "paged_attention: cudaFuncSetAttribute");
    CUtensorMap mk, mv;
    const bool f16 = E::kDtype == W4A16_DTYPE_F16;
    w4a16_status s = make_map(x.a.c, x.a.c.k, f16, x.box, &mk);
    if (s == W4A16_OK) s = make_map(x.a.c, x.a.c.v, f16, x.box, &mv);
    if (s != W4A16_OK) return s;
    return launch_overlapped("paged_attention", tile_kernel<E, D>, dim3((unsigned)dev.sms), kThreads, L::kSmem, st, mk,
                             mv, x);
}

}  // namespace

size_t attention_tile_workspace_bytes(const DeviceInfo& dev, int head_dim) {
    const size_t n = (size_t)dev.sms;
    return align_up(2 * n * sizeof(int)) + align_up(2 * n * kTile * sizeof(float2)) +
           2 * n * kTile * head_dim * sizeof(float);
}

w4a16_status attention_tile_launch(const DeviceInfo& dev, int dtype, const AttentionArgs& a, int min_rows,
                                   void* workspace, cudaStream_t st) {
    TileArgs x{};
    x.a = a;
    x.min_rows = min_rows;
    x.box = a.c.page_size & -a.c.page_size;
    if (x.box > kBlock) x.box = kBlock;
    unsigned char* w = static_cast<unsigned char*>(workspace);
    const size_t n = (size_t)dev.sms;
    x.counters = reinterpret_cast<int*>(w);
    w += align_up(2 * n * sizeof(int));
    x.stats = reinterpret_cast<float2*>(w);
    w += align_up(2 * n * kTile * sizeof(float2));
    x.parts = reinterpret_cast<float*>(w);
    const bool f16 = dtype == W4A16_DTYPE_F16;
    if (a.c.head_dim == 128) return f16 ? launch<Fp16, 128>(dev, x, st) : launch<Bf16, 128>(dev, x, st);
    return f16 ? launch<Fp16, 64>(dev, x, st) : launch<Bf16, 64>(dev, x, st);
}

#ifdef W4A16_TEST_HOOKS
cudaError_t attention_set_test_hooks(const TestHooks& h) { return cudaMemcpyToSymbol(g_hooks, &h, sizeof(h)); }
cudaError_t attention_get_test_counters(TestCounters* c) { return cudaMemcpyFromSymbol(c, g_counters, sizeof(*c)); }
#endif

}  // namespace w4a16
