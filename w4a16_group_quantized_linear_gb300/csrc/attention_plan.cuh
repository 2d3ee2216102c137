// Attention of new tokens over a paged cache: which kernel serves which sequences.
//
// A sequence's work is a number of rows per cached head: its new tokens times
// the query heads that share the head. With few rows the cache's bytes are all
// that counts and attention_step.cu takes them; past 16 the 8-row products
// of that kernel are what it waits for (with a variant for 32 rows, 25 rows of
// 16 sequences took 94 us, where the tiles take 87, and 32 of 64 sequences 132
// against 130), and attention_tile.cu takes 256 rows to a tile on the tensor
// cores. Over an 8-bit cache the tiles' conversion costs more than reading half as many bytes two or
// three times: there the step kernel takes up to 48 rows, in groups of 16 side by side. Measured on
// heads of 128, 5 to a cached one, of 16 sequences of 2000 to 9000 places alone: 25 rows 93 us and 143 in
// tiles, 45 rows 129 and 150 (bf16 94 and 167, 131 and 184).
//
// The lengths are on the device, so where a batch may hold both kinds both kernels are launched, and each
// passes over the other's. The step kernel's groups are then as many as max_q_len asks for, whether the
// batch has rows for them or not, and share the thread blocks evenly: 63 single tokens of 8 cached heads beside a
// chunk of 512 tokens take 449 us over 8 bits, 109 and 82 each alone, 264 over 16 bits.
#pragma once

#include "attention.cuh"

namespace w4a16 {

struct Plan {
    bool step, tile;
    int step_rows;  // most rows of a sequence of the step kernel
};

// most_rows: of a sequence of the step kernel.
inline Plan plan_for(int64_t T, int64_t batch, int heads, int kv_heads, int64_t max_q_len, int most_rows) {
    const int64_t ratio = heads / kv_heads, most = (max_q_len < T ? max_q_len : T) * ratio;
    Plan p;
    p.tile = most > most_rows;
    // every sequence has max_q_len new tokens, as one alone has: no second kind
    const bool alike = T == batch * max_q_len || batch == 1;
    p.step = !p.tile || (ratio <= most_rows && !alike);
    p.step_rows = (int)(most < most_rows ? most : most_rows);
    return p;
}

}  // namespace w4a16
