// Attention over the paged cache for many rows (chunks of new tokens): tiles of
// 256 rows, a row being one query head of one new token and the rows of a tile
// sharing one cached head, against blocks of 128 places on the tensor cores
// (sm_103a: TMA, tcgen05 MMA, TMEM).
//
// One pass over the places with the running maximum m and sum l of the
// softmax: p = 2^(c s - m), l += sum p, o = o 2^(m - m') + p v whenever m moves
// to m', which in whole tiles it only does when a score passes it by kMaxSlack
// (which keeps p inside the element type and makes the read-scale-write of o
// rare; out = o / l whatever m is).
//
// 4 D operations per (row, place) bound it: per block of 128 places and
// half tile of 128 rows two 128 x 128 x D products, 512 cycles each at D = 128,
// against 128 exponentials per row. The two halves of a tile take turns: while
// one half's scores go through the softmax, the tensor core forms the other's
// products, and each k and v block that is read serves 256 rows.
//
// Measured: 2048 tokens over 30048 places, 40 heads of 128 on 8: 786 to 805 us in short
// runs, 1510 to 1550 TFLOP/s, 79 to 81% of the cuBLAS bf16 burst (2900 cycles for a block of
// both halves, 2048 of them products); for seconds on end the power limit takes the clock to
// 1.6 GHz and it is 900 to 930 us. Heads of 64 have half the products to the same
// softmax: 633 us, 961 TFLOP/s. 14 sequences, 8 of single tokens, 6 of 287 to
// 1427 with a window of 1024, 32 heads of 64 on 4: 135 to 165 us from process to
// process, with the step kernel's 10. 5 tokens of 16 sequences over 2000 to 9000 places: 87 us.
//
//   warps 0-3, 4-7  softmax of the two halves: thread = row = TMEM lane. Reads
//                   its 128 scores (tcgen05.ld), writes p as 16-bit pairs over
//                   the first half of the same columns, where the second
//                   product takes it as its A operand. Also fetches its half's
//                   queries (rows of different tokens and heads: cp.async into the
//                   swizzled layout) while the last block of the tile before
//                   it is in work, and writes the result.
//   warps 8, 11     TMA: k blocks (8) and v blocks (11) into one ring of shared memory, the
//                   ring's even and odd entries, one box per page piece and 64
//                   elements. Pages that hold nothing to see are not read (a box outside
//                   the cache reads as zeros). Slots past a sequence's last place and
//                   before a window's first are zeroed in the v block (0 times whatever
//                   they hold might not be 0). Each warp waits for all entries in order: a
//                   barrier's parity tells only its next phase from the one before.
//   warp 9          MMA issue: p v of block j, then q k of block j + 1, for one half
//                   and then the other.
//   warp 10         lays out the work: each tile's rows, blocks and sharers, a few tiles
//                   ahead, so that the others keep none of it in registers.
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
constexpr int kLoadK = 8, kMmaWarp = 9, kPlanWarp = 10, kLoadV = 11;
constexpr int kBarBytes = 1792;  // struct Bars
constexpr int kEntries = 4;      // tiles of the work that are laid out ahead
// How far (log2) a score may pass the running maximum of a whole tile before the maximum moves. A
// weight reaches 2^14, inside fp16's 2^16, and o, not divided by l yet, that many times the values'
// sum: with bf16's range it has to stay small. (2^40 was no faster, and lost values past 2^87.)
constexpr float kMaxSlack = 14.0f;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOutCol = 256;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 1000000000ull;

#ifdef W4A16_TEST_HOOKS
__device__ TestHooks g_hooks = {kWaitLimitNs, -1};
__device__ TestCounters g_counters = {0ull, 0ull};
__device__ __forceinline__ uint64_t wait_limit() { return g_hooks.wait_limit_ns; }
__device__ __forceinline__ bool may_issue(int issued) {
    return g_hooks.issue_limit < 0 || issued < g_hooks.issue_limit;
}
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
    static constexpr int kSmem = kBarsAt + kBarBytes + 1024;  // barriers, and the 1024-byte alignment
};

constexpr int kMaxStages = 12;

// A tile, or a stretch of its blocks, for the warps to work on.
struct Entry {
    int b, g, first, count, length;
    int low;                   // first place that any row of the tile sees
    int from, to;              // blocks
    int ordinal;               // how many blocks of the run come before them
    int begin[2], end[2];      // of them, those of the halves: every one from begin to end, or every other
    int paired;                // the halves have the same rows and take turns with the blocks
    int c0, c1;                // the thread blocks that share the tile
    int last;
    int row;                   // first row of the tile
};

struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages];  // ring
    uint64_t landed;      // a v block that holds a sequence's last place or a window's first, before it is cleaned
    uint64_t q_full[2];   // a half's queries are in shared memory
    uint64_t s_full[2];   // a half's scores are in TMEM (and its o is up to date)
    uint64_t p_part[2];   // the first 64 columns of a half's p are in TMEM
    uint64_t p_full[2];   // and all of it
    uint64_t o_done[2];   // a half's o is complete for the tile
    uint64_t pair_in;     // the first half of a paired tile has left its o and statistics
    uint64_t pair_out;    // and the second has taken them
    uint64_t part_in[2];  // a half's threads have written their part
    uint64_t part_out[2]; // whether it was the last of its tile is known
    uint64_t work_full[kEntries], work_empty[kEntries];
    uint64_t mma_done;
    Entry work[kEntries];
    float2 pair_stats[kHalf];
    uint32_t tmem;
    int abort;
    int last[2];
};
static_assert(sizeof(Bars) <= kBarBytes, "barriers");

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
    const int first = __ldg(a.c.q_offsets + b), next = __ldg(a.c.q_offsets + b + 1), length = __ldg(a.c.kv_lens + b);
    s.first = first;
    s.count = next - first;
    s.tiles = 0;
    if (first < 0 || next > a.c.T || s.count <= 0 || s.count > a.max_q_len || s.count * a.ratio < x.min_rows) return;
    s.length = cache_length(a.c, length);
    s.tiles = (s.count * a.ratio + kTile - 1) / kTile;
}

// The places that rows [r0, r1) of a sequence see together, and their blocks.
struct Range {
    int low, block, end;  // block == end: none
};

__device__ __forceinline__ Range range_of(const AttentionArgs& a, int count, int length, int r0, int r1) {
    Range r{0, 0, 0};
    r1 = min(r1, count * a.ratio);
    if (r0 >= r1) return r;
    const int first = length - count + a.by_ratio.quotient(r0), last = length - count + a.by_ratio.quotient(r1 - 1);
    const int high = a.causal ? min(length, last + 1) : length;
    if (high <= 0) return r;
    r.low = first_seen(a, first);
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
    // with no second half of rows, and blocks enough, both halves work on the first
    __device__ __forceinline__ bool paired(int ratio) const {
        return s.count * ratio <= tile * kTile + kHalf && end - block > 1;
    }
};

__device__ __forceinline__ void set_tile(const AttentionArgs& a, Segment& s) {
    const int r = s.tile * kTile;
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

// Waits for the phase with the given parity, as ptx::mbar_wait does, but looks
// at the clock and the abort flag only every 32 polls: a read of the timer
// takes longer than a warp's share of a block may.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    uint64_t since = 0;
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (ptx::mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        const uint64_t now = ptx::globaltimer_ns();
        if (since == 0) since = now;
        else if (now - since > limit_ns) return false;
    }
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

// Slots of a block's last page piece that are past the sequence's `past` places in the block.
__device__ __forceinline__ int tail_rows(int past, int box) {
    return past > 0 && past < kBlock ? (box - (past & (box - 1))) & (box - 1) : 0;  // box: a power of two
}

// Slots of a block's first page piece to be read that are before the first place that a row of the
// tile sees, which is `before` places into the block.
__device__ __forceinline__ int head_rows(int before, int box) {
    return before > 0 && before < kBlock ? before & (box - 1) : 0;
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

// One lane of a converged warp, always the same one: true for it alone. (With a
// lane chosen by comparison the issue of one MMA took 115 cycles, not 64.)
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// Waits for this thread's TMEM loads, r's among them: as operands of the wait
// the registers cannot be read before it.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
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

struct Run {
    Shares shares;
    int64_t begin, end;
};

// The list's length, and where this thread block's run starts in it. All
// threads; scratch: 3 * kThreads ints of shared memory. Returns false where
// there is no run. Sequences a thread each, then their tiles a thread each;
// one round does for both questions while neither are more than the threads.
__device__ __forceinline__ bool find_run(const TileArgs& x, int* scratch, Run& run, Segment& at) {
    __shared__ int64_t s_sum[kThreads / 32];
    __shared__ int s_found[3];
    int* s_first = scratch;  // first tile of each of these sequences
    int* s_count = scratch + kThreads;
    int* s_length = s_count + kThreads;
    const AttentionArgs& a = x.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto share_out = [&](int64_t total) {
        run.shares.base = total / gridDim.x;
        run.shares.more = (int)(total - run.shares.base * gridDim.x);
        run.begin = run.shares.start(blockIdx.x);
        run.end = run.shares.start(blockIdx.x + 1);
    };
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
        int64_t before = 0;  // units of the tiles so far
#pragma unroll 1
        for (int b0 = 0; b0 < a.c.batch; b0 += kThreads) {
            Sequence s;
            s.tiles = 0;
            if (b0 + tid < a.c.batch) {
                load_sequence(x, b0 + tid, s);
                if (blockIdx.x == 0 && s.count > a.max_q_len) raise_device_error(a.c.err, W4A16_ERR_BAD_OFFSETS);
            }
            int tiles = 0;
            // what is summed: first the sequences' tiles, then the units of the tiles, kThreads at a time
#pragma unroll 1
            for (int i0 = -kThreads; i0 < tiles; i0 += kThreads) {
                int64_t n = s.tiles;
                int lo = 0, tile = 0;
                if (i0 >= 0) {
                    n = 0;
                    if (i0 + tid < tiles) {
                        int hi = kThreads - 1;  // the last sequence that starts at or before the tile
                        while (lo < hi) {
                            const int mid = (lo + hi + 1) >> 1;
                            if (s_first[mid] <= i0 + tid) lo = mid;
                            else hi = mid - 1;
                        }
                        Segment t;
                        tile = t.tile = i0 + tid - s_first[lo];
                        t.s.count = s_count[lo];
                        t.s.length = s_length[lo];
                        set_tile(a, t);
                        n = (int64_t)(t.end - t.block) * a.c.kv_heads;
                    }
                }
                int64_t upto = n;  // inclusive sum over the threads
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int64_t u = __shfl_up_sync(0xffffffffu, upto, d);
                    if (lane >= d) upto += u;
                }
                __syncthreads();
                if (lane == 31) s_sum[warp] = upto;
                __syncthreads();
                int64_t all = 0;
#pragma unroll 1
                for (int w = 0; w < kThreads / 32; ++w) {
                    if (w < warp) upto += s_sum[w];
                    all += s_sum[w];
                }
                if (i0 < 0) {
                    tiles = (int)all;
                    s_first[tid] = (int)(upto - n);
                    s_count[tid] = s.count;
                    s_length[tid] = s.length;
                    __syncthreads();
                    continue;
                }
                upto += before;
                before += all;
                if (round == 0 && a.c.batch <= kThreads && tiles <= kThreads) {
                    share_out(before);
                    round = 1;
                }
                if (round == 1 && n > 0 && run.begin >= upto - n && run.begin < upto) {
                    s_found[0] = b0 + lo;
                    s_found[1] = tile;
                    s_found[2] = (int)(run.begin - (upto - n));
                }
            }
            __syncthreads();
            if (round == 1 && before > run.begin) break;
        }
        if (round == 0) share_out(before);
        if (run.begin >= run.end) return false;
    }
    at.b = s_found[0];
    at.tile = s_found[1];
    load_sequence(x, at.b, at.s);
    set_tile(a, at);
    at.g = s_found[2] / (at.end - at.block);
    at.from = at.block + s_found[2] % (at.end - at.block);
    at.to = (int)min((int64_t)at.end, at.from + (run.end - run.begin));
    return true;
}

template <class E, int D, bool PAIRED>
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
    const int ratio = a.ratio;

    // what does not depend on the kernel before this one
    if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < L::kStages; ++i) {
                ptx::mbar_init(&bars->full[i], 1);
                ptx::mbar_init(&bars->empty[i], 1);
            }
            for (int w = 0; w < 2; ++w) {
                ptx::mbar_init(&bars->q_full[w], kHalf);
                ptx::mbar_init(&bars->s_full[w], 1);
                ptx::mbar_init(&bars->p_part[w], kHalf / 32);
                ptx::mbar_init(&bars->p_full[w], kHalf / 32);
                ptx::mbar_init(&bars->o_done[w], 1);
                ptx::mbar_init(&bars->part_in[w], kHalf);
                ptx::mbar_init(&bars->part_out[w], 1);
            }
            for (int i = 0; i < kEntries; ++i) {
                ptx::mbar_init(&bars->work_full[i], 1);
                ptx::mbar_init(&bars->work_empty[i], PAIRED ? 12 : 11);  // loads, MMAs (of each half), softmax warps
            }
            ptx::mbar_init(&bars->landed, 1);
            ptx::mbar_init(&bars->pair_in, kHalf);
            ptx::mbar_init(&bars->pair_out, kHalf);
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
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (blockIdx.x == 0) check_offsets(a.c);
    Run run;
    Segment seg;
    bool ok = find_run(x, reinterpret_cast<int*>(ring), run, seg);  // false, for all threads: nothing to do
    ptx::fence_proxy_async_shared();  // the scratch above was the ring's memory
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = bars->tmem;
    volatile int* abort = &bars->abort;
    const bool idle = !ok;
    // entry k of the work, for this warp to read; false if it gave up
    auto entry = [&](int k) {
        if (ok && !wait_bar(&bars->work_full[k % kEntries], (k / kEntries) & 1, abort, wait_limit())) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        return ok;
    };
    auto done_with = [&](int k) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->work_empty[k % kEntries]);
    };

    if (idle) {
        // straight to the end
    } else if (warp == kPlanWarp) {
        // -------------------------------------------------------------- plan
        int64_t left = run.end - run.begin, unit = run.begin;
        for (int k = 0; ok; ++k) {
            if (k >= kEntries &&
                !wait_bar(&bars->work_empty[k % kEntries], (k / kEntries - 1) & 1, abort, wait_limit()))
                ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const int n = seg.to - seg.from;
            if (lane == 0) {
                Entry& e = bars->work[k % kEntries];
                e.b = seg.b;
                e.g = seg.g;
                e.row = seg.tile * kTile;
                e.first = seg.s.first;
                e.count = seg.s.count;
                e.length = seg.s.length;
                e.low = seg.low;
                e.from = seg.from;
                e.to = seg.to;
                e.ordinal = (int)(unit - run.begin);
                e.paired = PAIRED && seg.paired(ratio);
                e.begin[0] = max(seg.half0.block, seg.from);
                e.begin[1] = e.paired ? seg.from + 1 : max(seg.half1.block, seg.from);
                e.end[0] = min(seg.half0.end, seg.to);
                e.end[1] = e.paired ? e.end[0] : min(seg.half1.end, seg.to);
                const int64_t item = unit - (seg.from - seg.block);
                e.c0 = run.shares.owner(item, blockIdx.x);
                e.c1 = run.shares.owner(item + (seg.end - seg.block) - 1, blockIdx.x);
                e.last = left == n;
                ptx::mbar_arrive(&bars->work_full[k % kEntries]);
            }
            left -= n;
            unit += n;
            if (left == 0) break;
            next_segment(x, left, seg);
        }
        if (!ok && lane == 0) fail(x, bars);
    } else if (warp == kLoadK || warp == kLoadV) {
        // ------------------------------------------------------------- loads
        // k blocks are the ring's even entries, v blocks the odd ones
        const bool values = warp == kLoadV;
        const CUtensorMap* map = values ? &map_v : &map_k;
        const int pieces = kBlock / x.box;
        const int piece = lane / L::kSlabs, slab = lane % L::kSlabs;
        int n = 0, issued = -1;
        // The v block of a sequence's last place, or of a window's first, lands on a barrier
        // of its own; then its slots past the one and before the other are zeroed (0 times what
        // they hold might not be 0), and only then is it handed on. Other copies go out meanwhile,
        // but nothing is waited for before that.
        int dirty = -1, dirty_head = 0, dirty_heads = 0, dirty_row = 0, dirty_rows = 0;
        uint32_t landed_parity = 0;
        auto clean = [&] {
            ok = ok && wait_bar(&bars->landed, landed_parity, abort, wait_limit());
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            landed_parity ^= 1u;
            const int st = dirty % L::kStages;
            for (int c = lane; c < (dirty_heads + dirty_rows) * (D / 8); c += 32) {
                const int i = c / (D / 8), part = c % (D / 8);
                const int row = i < dirty_heads ? dirty_head + i : dirty_row + i - dirty_heads;
                *reinterpret_cast<uint4*>(ring + st * L::kStageBytes + (part >> 3) * L::kSlabBytes + row * 128 +
                                          (part & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            ptx::fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bars->full[st]);
            dirty = -1;
        };
        auto wait_clean = [&](uint64_t* bar, uint32_t parity) {
            if (__all_sync(0xffffffffu, ok && ptx::mbar_try_wait(bar, parity))) return true;
            if (dirty >= 0) clean();
            ok = ok && wait_bar(bar, parity, abort, wait_limit());
            ok = __all_sync(0xffffffffu, ok);
            return ok;
        };
        for (int k = 0; wait_clean(&bars->work_full[k % kEntries], (k / kEntries) & 1); ++k) {
            const Entry& e = bars->work[k % kEntries];
            const int to = e.to, length = e.length, low = e.low, b = e.b, g = e.g;
            const bool last = e.last;
            // the pages of 32 pieces, a lane each, read a group ahead; outside the cache: zeros
            auto pages_from = [&](int first) {
                const int p = (first + lane) * x.box;
                int64_t page = -1;
                if (p < length && p + x.box > low && p < to * kBlock) page = page_of(a.c, b, p);
                return (int)(page < 0 ? a.c.pages : page);
            };
            int group = e.from * pieces;  // its first piece
            int pages = pages_from(group), more_pages = pages_from(group + 32);
            for (int j = e.from; ok && j < to; ++j) {
                if (j * pieces >= group + 32) {
                    group += 32;
                    pages = more_pages;
                    more_pages = pages_from(group + 32);
                }
                const int page = __shfl_sync(0xffffffffu, pages, j * pieces - group + (piece & (pieces - 1)));
                // Both of a block's stages are waited for in the ring's order, the other
                // warp's too: a barrier's parity tells only its next phase from the one before.
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++n) {
                    const int st = n % L::kStages, round = n / L::kStages;
                    if (dirty >= 0 && __all_sync(0xffffffffu, ptx::mbar_try_wait(&bars->landed, landed_parity)))
                        clean();
                    if (round > 0 && !wait_clean(&bars->empty[st], (round - 1) & 1)) break;
                    if (kv != (values ? 1 : 0)) continue;
                    ok = may_issue(n);
                    if (!ok) break;
                    const int rows = values ? tail_rows(length - j * kBlock, x.box) : 0;
                    const int heads = values ? head_rows(low - j * kBlock, x.box) : 0;
                    const bool unclean = rows + heads > 0;
                    if (unclean && dirty >= 0) {
                        clean();
                        if (!ok) break;
                    }
                    uint64_t* bar = unclean ? &bars->landed : &bars->full[st];
                    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, L::kStageBytes);
                    __syncwarp();
                    if (piece < pieces)
                        tma_load_4d(ring + st * L::kStageBytes + slab * L::kSlabBytes + piece * x.box * 128, map, bar,
                                    slab * 64, a.c.by_page.remainder(j * kBlock + piece * x.box), g, page);
                    issued = n;
                    if (unclean) {
                        dirty = n;
                        dirty_head = low - j * kBlock - heads;
                        dirty_heads = heads;
                        dirty_row = length - j * kBlock;
                        dirty_rows = rows;
                    }
                }
            }
            done_with(k);
            if (!ok || last) break;
        }
        if (ok && dirty >= 0) clean();
        if (!ok && lane == 0) {
            fail(x, bars);
            volatile int never = 0;  // our own copies land before the thread block ends
            if (dirty >= 0) wait_bar(&bars->landed, landed_parity, &never, kDrainLimitNs);
            for (int i = issued; i >= 0 && i > issued - L::kStages; i -= 2)
                if (i != dirty)
                    wait_bar(&bars->full[i % L::kStages], (i / L::kStages) & 1, &never, kDrainLimitNs);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // --------------------------------------------------------------- MMA
        // One thread. The tensor core's queue holds about 200 cycles of products, so what
        // this thread does between two of them is kept below that: what comes next is
        // worked out while products are queued, not at its turn.
        constexpr uint32_t kIdescS = idesc<E>(kBlock, false), kIdescO = idesc<E>(D, true);
        if (elect_one()) {
            const uint32_t ring_u = ptx::smem_u32(ring);
            const uint64_t q_desc = ptx::smem_desc_sw128(ptx::smem_u32(smem));
            const uint64_t k_desc = ptx::smem_desc_sw128(ring_u), v_desc = desc_v(ring_u, L::kSlabBytes);
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                if (!ptx::mbar_try_wait(bar, parity) && !wait_bar(bar, parity, abort, wait_limit())) ok = false;
                ptx::tc_fence_after();
                return ok;
            };
            auto scores = [&](int w, uint32_t st) {
                const uint64_t q = q_desc + (uint64_t)(w * (L::kStageBytes >> 4));
                const uint64_t k = k_desc + (uint64_t)(st * (L::kStageBytes >> 4));
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint64_t at = (uint64_t)(((ks >> 2) * L::kSlabBytes + (ks & 3) * 32) >> 4);
                    mma_ss(tmem + w * kBlock, q + at, k + at, kIdescS, ks > 0);
                }
                ptx::mma_commit(&bars->s_full[w]);
            };
            // p v; where p is not complete yet, the first half of the contraction goes ahead
            auto output = [&](int w, uint32_t st, uint32_t parity, bool first, bool last) {
                const uint64_t v = v_desc + (uint64_t)(st * (L::kStageBytes >> 4));
                const uint32_t o = tmem + kOutCol + w * D, p = tmem + w * kBlock;
                if (!wait(&bars->p_part[w], parity)) return false;
                ptx::mma_f16_ts(o, p, v, kIdescO, !first);
#pragma unroll
                for (int kk = 1; kk < kBlock / 32; ++kk)
                    ptx::mma_f16_ts(o, p + kk * 8, v + (uint64_t)((kk * 2048) >> 4), kIdescO, 1u);
                if (!wait(&bars->p_full[w], parity)) return false;
#pragma unroll
                for (int kk = kBlock / 32; kk < kBlock / 16; ++kk)
                    ptx::mma_f16_ts(o, p + kk * 8, v + (uint64_t)((kk * 2048) >> 4), kIdescO, 1u);
                if (last) ptx::mma_commit(&bars->o_done[w]);
                return true;
            };
            if constexpr (!PAIRED) {
                // Block by block, one half and then the other.
                // what a block needs of its entry
                struct View {
                    int to, begin0, end0, begin1, end1, last;
                };
                auto view = [&](int k) {
                    const Entry& e = bars->work[k % kEntries];
                    return View{e.to, e.begin[0], e.end[0], e.begin[1], e.end[1], e.last};
                };
                auto advance = [](uint32_t& st, uint32_t& parity) {
                    if (++st == L::kStages) {
                        st = 0;
                        parity ^= 1u;
                    }
                };
                int k = 0;                                // entry of the block whose p v comes next
                int j = 0, i = 0;                         // that block, and the one whose scores come next
                uint32_t vst = 0, vparity = 0, kst = 0, kparity = 0;  // their ring stages
                uint32_t q_parity0 = 0, q_parity1 = 0, p_parity0 = 0, p_parity1 = 0;
                bool turn = false, more = true;           // the two are of different entries; there is a second one
                View cur{}, nxt{};
                auto plan = [&] {
                    vst = kst;
                    vparity = kparity;
                    advance(vst, vparity);
                    kst = vst;
                    kparity = vparity;
                    advance(kst, kparity);
                    i = j + 1;
                    turn = i == cur.to;
                    more = !turn || !cur.last;
                    if (turn && more && wait(&bars->work_full[(k + 1) % kEntries], ((k + 1) / kEntries) & 1)) {
                        nxt = view(k + 1);
                        i = bars->work[(k + 1) % kEntries].from;
                    }
                };
                if (wait(&bars->work_full[0], 0)) {  // the first block's scores
                    cur = nxt = view(0);
                    j = bars->work[0].from;
                    wait(&bars->full[0], 0);
                    if (ok && j >= cur.begin0 && j < cur.end0 && wait(&bars->q_full[0], 0)) {
                        scores(0, 0);
                        q_parity0 = 1;
                    }
                    if (ok && j >= cur.begin1 && j < cur.end1 && wait(&bars->q_full[1], 0)) {
                        scores(1, 0);
                        q_parity1 = 1;
                    }
                    ptx::mma_commit(&bars->empty[0]);
                    plan();
                }
                while (ok) {
                    if (!wait(&bars->full[vst], vparity)) break;
                    if (j >= cur.begin0 && j < cur.end0) {
                        if (!output(0, vst, p_parity0, j == cur.begin0, j == cur.end0 - 1)) break;
                        p_parity0 ^= 1u;
                    }
                    if (more) {
                        if (!wait(&bars->full[kst], kparity)) break;
                        if (i >= nxt.begin0 && i < nxt.end0) {
                            if (i == nxt.begin0) {
                                if (!wait(&bars->q_full[0], q_parity0)) break;
                                q_parity0 ^= 1u;
                            }
                            scores(0, kst);
                        }
                    }
                    if (j >= cur.begin1 && j < cur.end1) {
                        if (!output(1, vst, p_parity1, j == cur.begin1, j == cur.end1 - 1)) break;
                        p_parity1 ^= 1u;
                    }
                    ptx::mma_commit(&bars->empty[vst]);
                    if (!more) break;
                    // the round after this one, while the products above are queued
                    const bool second = i >= nxt.begin1 && i < nxt.end1;
                    if (second && i == nxt.begin1) {
                        if (!wait(&bars->q_full[1], q_parity1)) break;
                        q_parity1 ^= 1u;
                    }
                    const uint32_t st = kst;
                    if (turn) {
                        ptx::mbar_arrive(&bars->work_empty[k % kEntries]);
                        ++k;
                        cur = nxt;
                    }
                    j = i;
                    plan();
                    if (!ok) break;
                    if (second) scores(1, st);
                    ptx::mma_commit(&bars->empty[st]);
                }
            } else {
                // The two halves are two streams of blocks: each has its next scores formed as
                // soon as its last p is used up. The one that is further behind goes first, and neither
                // passes the other by more than two blocks. Every block of the run is waited
                // for by each, in order, whether the half sees it or not.
                //
                // A half's p may depend on what the other has yet to do: at the end of a paired
                // tile each waits for the other's o (pair_in, pair_out) before its next p, and
                // the stream ahead may be in the tile after that. So nothing is waited for here
                // that is not on its way whatever this thread does: the first part of p is polled
                // for like all else (its second part follows from the same pass). The stream
                // behind can always go on, and that is enough: all of the other's products of the tiles
                // before it are issued, so its half gets past them, fetches its queries and
                // announces p; and its blocks are loaded, as the ring holds the two blocks that the
                // other may be ahead.
                struct Stream {
                    int k = -1, j = 0, to = 0;          // entry, block, and the end of the entry's blocks
                    int begin = 0, end = 0, step = 1;   // the half's blocks of the entry
                    int shift = 0;                      // from block to place in the run
                    bool last = false, more = true;
                    bool formed = false;                // the block's scores are on their way
                    uint32_t q_parity = 0, p_parity = 0;
                    __device__ __forceinline__ int at() const { return j + shift; }
                } s0, s1;
                // gives a ring entry back, if the other stream is through with it too (else it will)
                auto release = [&](int n, const Stream& other) {
                    if (other.at() > n >> 1 || (other.at() == n >> 1 && other.formed && !(n & 1)))
                        ptx::mma_commit(&bars->empty[n % L::kStages]);
                };
                auto here = [&](int n) {  // entry n of the ring has landed
                    return ptx::mbar_try_wait(&bars->full[n % L::kStages], (n / L::kStages) & 1);
                };
                // towards the half's next block, as far as that goes without waiting
                auto advance = [&](int w, Stream& s, const Stream& other) {
                    bool moved = false;
                    while (s.more && !s.formed) {
                        if (s.j == s.to) {
                            if (s.last) {
                                ptx::mbar_arrive(&bars->work_empty[s.k % kEntries]);
                                s.more = false;
                                return true;
                            }
                            const int k = s.k + 1;
                            if (!ptx::mbar_try_wait(&bars->work_full[k % kEntries], (k / kEntries) & 1)) return moved;
                            if (k > 0) ptx::mbar_arrive(&bars->work_empty[s.k % kEntries]);
                            const Entry& e = bars->work[k % kEntries];
                            s.k = k;
                            s.j = e.from;
                            s.to = e.to;
                            s.begin = e.begin[w];
                            s.end = e.end[w];
                            s.step = e.paired ? 2 : 1;
                            s.shift = e.ordinal - e.from;
                            s.last = e.last;
                            moved = true;
                        }
                        const int n = 2 * s.at();
                        if ((other.more && s.at() > other.at() + 2) || !here(n)) return moved;
                        if (s.j >= s.begin && s.j < s.end && ((s.j - s.begin) & (s.step - 1)) == 0) {
                            if (s.j == s.begin) {
                                if (!ptx::mbar_try_wait(&bars->q_full[w], s.q_parity)) return moved;
                                s.q_parity ^= 1u;
                            }
                            ptx::tc_fence_after();
                            scores(w, n % L::kStages);
                            release(n, other);
                            s.formed = true;
                            return true;
                        }
                        if (!here(n + 1)) return moved;
                        release(n, other);
                        release(n + 1, other);
                        ++s.j;
                        moved = true;
                    }
                    return moved;
                };
                auto add_values = [&](int w, Stream& s, const Stream& other) {
                    const int n = 2 * s.at() + 1;
                    if (!here(n)) return false;
                    // Where the half goes on in the same tile and the blocks up to its next one are
                    // here, that is found out before the wait for p, and the next scores follow
                    // the products at once.
                    const int ahead = n - 1 + 2 * s.step;  // the next block's k
                    bool on = s.j + s.step < s.end && (!other.more || s.at() + s.step <= other.at() + 2) && here(ahead);
                    if (s.step == 2) on = on && here(n + 1) && here(n + 2);
                    const int st = ahead % L::kStages;
                    if (!ptx::mbar_try_wait(&bars->p_part[w], s.p_parity)) return false;
                    if (!output(w, n % L::kStages, s.p_parity, s.j == s.begin, s.j + s.step >= s.end)) return false;
                    s.p_parity ^= 1u;
                    release(n, other);
                    if (on) scores(w, st);
                    if (on) {
                        if (s.step == 2) {
                            release(n + 1, other);
                            release(n + 2, other);
                        }
                        release(ahead, other);
                        s.j += s.step;
                    } else {
                        ++s.j;
                        s.formed = false;
                    }
                    return true;
                };
                uint64_t since = 0;
                int idle = 0;
                while (ok && (s0.more || s1.more)) {
                    bool moved = s0.formed && (!s1.formed || s0.at() <= s1.at()) && add_values(0, s0, s1);
                    if (!moved && s1.formed) moved = add_values(1, s1, s0);
                    moved |= advance(0, s0, s1);
                    moved |= advance(1, s1, s0);
                    if (moved) {
                        idle = 0;
                        since = 0;
                    } else if ((++idle & 31) == 0) {  // bounded, like every wait
                        const uint64_t now = ptx::globaltimer_ns();
                        if (since == 0) since = now;
                        if (*abort || now - since > wait_limit()) ok = false;
                    }
                }
            }
            if (!ok) fail(x, bars);
            ptx::mma_commit(&bars->mma_done);
            volatile int never = 0;
            wait_bar(&bars->mma_done, 0, &never, kDrainLimitNs);
        }
        __syncwarp();
    } else {
        // ----------------------------------------------------------- softmax
        // How far a score may pass the maximum before it moves. Not at all where there are few rows,
        // whose time is the cache's: the largest weight is then 1 and exact, and the error of
        // rounding p next to nothing (87 against 85 us at 25 rows; errors 1.0 to 1.1 times
        // that of rounding the result alone, where they are up to 1.7 times). For whole tiles
        // it would cost 11% (2048 tokens over 30048 places 870 against 786 us) for errors of
        // 1.1 instead of 1.4 times.
        constexpr float kSlack = PAIRED ? 0.0f : kMaxSlack;
        const int w = warp >> 2;
        const int row = tid & (kHalf - 1);
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_addr = lane_base + w * kBlock, o_addr = lane_base + kOutCol + w * D;
        const uint32_t q_smem = ptx::smem_u32(smem) + w * L::kStageBytes;
        int ns = 0, no = 0, nj = 0, npair = 0;
        // this half's queries of an entry, 16 bytes a lane; rows past the sequence's are zeros
        auto load_q = [&](const Entry& e) {
            constexpr int kPieces = D / 8, kRowsPer = 32 / kPieces;
            const int piece = lane % kPieces;
#pragma unroll 4
            for (int i = 0; i < 32 / kRowsPer; ++i) {
                const int r = (warp & 3) * 32 + i * kRowsPer + lane / kPieces;
                const int at = e.row + (PAIRED && e.paired ? 0 : w * kHalf) + r;
                const int token = a.by_ratio.quotient(at);
                const bool real = token < e.count;
                const uint16_t* src =
                    a.q + (real ? (e.first + token) * a.q_row_stride +
                                      (int64_t)(e.g * ratio + at - token * ratio) * a.q_head_stride + piece * 8
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
        if (entry(0) && bars->work[0].end[w] > bars->work[0].begin[w]) {
            load_q(bars->work[0]);
            q_ready();
        }
        for (int k = 0; ok; ++k) {
            const Entry& e = bars->work[k % kEntries];
            const Entry& next = bars->work[(k + 1) % kEntries];
            const bool last = e.last;
            const bool paired = PAIRED && e.paired;
            const int begin = e.begin[w], end = e.end[w], step = paired ? 2 : 1;
            const int first_row = e.row + (paired ? 0 : w * kHalf);
            int low, high;
            {
                const int token = a.by_ratio.quotient(first_row + row);
                const int place = e.length - e.count + token;
                low = first_seen(a, place);
                high = token >= e.count ? 0 : a.causal ? min(e.length, place + 1) : e.length;
            }
            bool load_next = false;
            float m = -INFINITY;
            float2 sum = make_float2(0.0f, 0.0f);
            for (int j = begin; j < end; j += step) {
                if (!wait_bar(&bars->s_full[w], ns & 1, abort, wait_limit())) ok = false;
                ++ns;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ptx::tc_fence_after();
                if (j + step >= end && !last) {  // the last scores are formed: q may go
                    if (!entry(k + 1)) break;
                    load_next = next.end[w] > next.begin[w];
                    if (load_next) load_q(next);
                }
                // The scores are read twice, for the maximum and for p, the second time 32
                // columns at a time in a loop: straight code for them all is longer than the
                // instruction cache that the issuing warp shares. Blocks at the edge of what
                // a row sees are masked in place first.
                const int lo = low - j * kBlock, hi = high - j * kBlock;
                if (__any_sync(0xffffffffu, lo > 0 || hi < kBlock)) {
#pragma unroll 1
                    for (int c = 0; c < kBlock; c += 32) {
                        if (!__any_sync(0xffffffffu, lo > c || hi < c + 32)) continue;
                        uint32_t s[32];
                        ptx::tmem_ld_32x32b_x32(s_addr + c, s);
                        tmem_ld_wait(s);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i < lo || c + i >= hi) s[i] = 0xFF800000u;  // -infinity
                        ptx::tmem_st_32x32b_x32(s_addr + c, s);
                    }
                    ptx::tmem_st_wait();
                }
                uint32_t s0[32], s1[32];
                float t[4];
                ptx::tmem_ld_32x32b_x32(s_addr, s0);
                ptx::tmem_ld_32x32b_x32(s_addr + 32, s1);
                tmem_ld_wait(s0);
                tmem_ld_wait(s1);
#pragma unroll
                for (int i = 0; i < 4; ++i) t[i] = __uint_as_float(s0[i]);
                auto largest = [&](const uint32_t (&s)[32]) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            t[u] = max3(t[u], __uint_as_float(s[i + 2 * u]), __uint_as_float(s[i + 2 * u + 1]));
                };
                largest(s0);
                ptx::tmem_ld_32x32b_x32(s_addr + 64, s0);
                largest(s1);
                ptx::tmem_ld_32x32b_x32(s_addr + 96, s1);
                tmem_ld_wait(s0);
                tmem_ld_wait(s1);
                largest(s0);
                ptx::tmem_ld_32x32b_x32(s_addr, s0);
                largest(s1);
                float top = fmaxf(max3(t[0], t[1], t[2]), t[3]) * a.scale_log2;
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
                auto weights = [&](int c, uint32_t (&s)[32]) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 v = fma2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c2, m2);
                        v.x = fast_exp2(v.x);
                        v.y = fast_exp2(v.y);
                        sum = add2(sum, v);
                        p[i] = E::pack(v.x, v.y);
                    }
                    ptx::tmem_st_32x32b_x16(s_addr + (c >> 1), p);
                };
#pragma unroll 1
                for (int c = 0; c < kBlock; c += 64) {
                    tmem_ld_wait(s0);
                    ptx::tmem_ld_32x32b_x32(s_addr + c + 32, s1);
                    weights(c, s0);
                    tmem_ld_wait(s1);
                    ptx::tmem_ld_32x32b_x32(s_addr + 64, s0);  // (the last time for nothing)
                    weights(c + 32, s1);
                    ptx::tmem_st_wait();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(c == 0 ? &bars->p_part[w] : &bars->p_full[w]);
                }
                tmem_ld_wait(s0);
            }
            if (!ok) break;
            if (begin >= end && !last) {
                if (!entry(k + 1)) break;
                load_next = next.end[w] > next.begin[w];
                if (load_next) load_q(next);
            }
            if (load_next) q_ready();
            // ---- the tile's result, or this thread block's part of it
            if (end > begin) {
                if (!wait_bar(&bars->o_done[w], no & 1, abort, wait_limit())) ok = false;
                ++no;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ptx::tc_fence_after();
            }
            float l = sum.x + sum.y;
            // A paired tile: the second half adds the first one's o, straight from its TMEM columns.
            float scale = 1.0f, scale0 = 0.0f;
            if (paired) {
                if (w == 0) {
                    bars->pair_stats[row] = make_float2(m, l);
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(&bars->pair_in);
                }
                if (!wait_bar(w == 0 ? &bars->pair_out : &bars->pair_in, npair & 1, abort, wait_limit())) ok = false;
                ++npair;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ptx::tc_fence_after();
                if (w == 0) {
                    done_with(k);
                    if (last) break;
                    continue;
                }
                const float2 other = bars->pair_stats[row];
                const float top = fmaxf(m, other.x);
                scale = m == -INFINITY ? 0.0f : fast_exp2(m - top);
                scale0 = other.x == -INFINITY ? 0.0f : fast_exp2(other.x - top);
                m = top;
                l = l * scale + other.y * scale0;
            }
            const int at = first_row + row;
            const int token = a.by_ratio.quotient(at);
            const bool real = token < e.count;
            const int64_t out_row = (int64_t)(e.first + token) * a.heads + e.g * ratio + at - token * ratio;
            const int c0 = e.c0, c1 = e.c1;
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
            const int64_t slot = 2 * (int64_t)blockIdx.x + (c0 == (int)blockIdx.x ? 1 : 0);
            const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
                uint32_t r[32];
                float v[32];
                if (end > begin) {
                    ptx::tmem_ld_32x32b_x32(o_addr + d, r);
                    tmem_ld_wait(r);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = end > begin ? __uint_as_float(r[i]) * scale : 0.0f;
                if (paired) {
                    ptx::tmem_ld_32x32b_x32(o_addr - D + d, r);
                    tmem_ld_wait(r);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] += __uint_as_float(r[i]) * scale0;
                }
                if (c0 == c1) {
                    if (real) write32(d, v, inv);
                } else {
                    float* dst = x.parts + (slot * D + d) * kTile + w * kHalf + row;
#pragma unroll
                    for (int i = 0; i < 32; ++i) __stcg(dst + i * kTile, v[i]);
                }
            }
            ptx::tc_fence_before();  // o may be overwritten once the next p is announced
            if (paired) ptx::mbar_arrive(&bars->pair_out);
            if (c0 == c1) {
                if (real) write_lse(m, l);
            } else {
                __stcg(x.stats + slot * kTile + w * kHalf + row, make_float2(m, l));
                __threadfence();
                ptx::mbar_arrive(&bars->part_in[w]);
                int* counter = x.counters + 2 * c0 + w;
                if (row == 0 && wait_bar(&bars->part_in[w], nj & 1, abort, wait_limit())) {
                    const int done = ptx::atom_add_acq_rel_gpu(counter, 1);
                    bars->last[w] = done == c1 - c0;
                    if (bars->last[w]) *counter = 0;
                    ptx::mbar_arrive(&bars->part_out[w]);
                }
                __syncwarp();
                if (!wait_bar(&bars->part_out[w], nj & 1, abort, wait_limit())) ok = false;
                ++nj;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (bars->last[w]) {
                    __threadfence();
                    // of thread blocks c0 to c1: the first one's last tile, the others' first
                    const int parts = c1 - c0 + 1;
                    auto slot_of = [&](int i) { return (int64_t)(2 * (c0 + i) + (i == 0)); };
                    auto stats = [&](int i) { return __ldcg(x.stats + slot_of(i) * kTile + w * kHalf + row); };
                    float top = -INFINITY, total = 0.0f;
#pragma unroll 4
                    for (int i = 0; i < parts; ++i) top = fmaxf(top, stats(i).x);
#pragma unroll 4
                    for (int i = 0; i < parts; ++i) {
                        const float2 v = stats(i);
                        total += v.y * (v.x == -INFINITY ? 0.0f : fast_exp2(v.x - top));  // a sum of NaN stays one
                    }
                    const float inv_total = total > 0.0f || total != total ? 1.0f / total : 0.0f;
#pragma unroll 1
                    for (int d = 0; d < D; d += 32) {
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0.0f;
#pragma unroll 2
                        for (int i = 0; i < parts; ++i) {
                            const float mc = stats(i).x;
                            const float f = mc == -INFINITY ? 0.0f : fast_exp2(mc - top);
                            const float* src = x.parts + (slot_of(i) * D + d) * kTile + w * kHalf + row;
#pragma unroll
                            for (int c = 0; c < 32; ++c) v[c] += f * __ldcg(src + c * kTile);
                        }
                        if (real) write32(d, v, inv_total);
                    }
                    if (real) write_lse(top, total);
                }
            }
            done_with(k);
            if (last) break;
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

template <class E, int D, bool PAIRED>
w4a16_status launch(const DeviceInfo& dev, const TileArgs& x, cudaStream_t st) {
    using L = Layout<D>;
    static_assert(L::kStages <= kMaxStages, "ring");
    static PerDeviceOnce once;
    const cudaError_t e = once.run(dev.device, [] {
        return cudaFuncSetAttribute(tile_kernel<E, D, PAIRED>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    });
    if (e != cudaSuccess) return cuda_status(e, "paged_attention: cudaFuncSetAttribute");
    CUtensorMap mk, mv;
    const bool f16 = E::kDtype == W4A16_DTYPE_F16;
    w4a16_status s = make_map(x.a.c, x.a.c.k, f16, x.box, &mk);
    if (s == W4A16_OK) s = make_map(x.a.c, x.a.c.v, f16, x.box, &mv);
    if (s != W4A16_OK) return s;
    return launch_overlapped("paged_attention", tile_kernel<E, D, PAIRED>, dim3((unsigned)dev.sms), kThreads, L::kSmem,
                             st, mk, mv, x);
}

template <class E, int D>
w4a16_status launch_rows(const DeviceInfo& dev, const TileArgs& x, cudaStream_t st) {
    // Sequences that all fit half a tile (drafts being verified, short chunks)
    // share out their blocks between the halves: 5 tokens x 5 heads over 2000 to
    // 9000 places, 16 sequences, 87 us against 103 with one half idle (and the
    // maximum that lags). For tiles of both halves the issuing loop that
    // knows of no pairs is the faster one (2048 tokens over 30048 places 807
    // against 868 us when both were built with that maximum).
    return x.a.max_q_len * x.a.ratio <= kHalf ? launch<E, D, true>(dev, x, st) : launch<E, D, false>(dev, x, st);
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
    if (a.c.head_dim == 128) return f16 ? launch_rows<Fp16, 128>(dev, x, st) : launch_rows<Bf16, 128>(dev, x, st);
    return f16 ? launch_rows<Fp16, 64>(dev, x, st) : launch_rows<Bf16, 64>(dev, x, st);
}

#ifdef W4A16_TEST_HOOKS
cudaError_t attention_set_test_hooks(const TestHooks& h) { return cudaMemcpyToSymbol(g_hooks, &h, sizeof(h)); }
cudaError_t attention_get_test_counters(TestCounters* c) { return cudaMemcpyFromSymbol(c, g_counters, sizeof(*c)); }
#endif

}  // namespace w4a16
