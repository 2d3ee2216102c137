// Rotary positions as the kernels that turn heads see them: the angle table, the
// positions, and the 16 elements of 8 pairs that a thread takes.
#pragma once

#include "attention.cuh"

namespace w4a16 {

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

// ------------------------------------------------------------------ host --

inline void fill(RotaryArgs& r, const w4a16_rotary* rotary) {
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

}  // namespace w4a16
