"""Rotary positions, the paged cache and attention over it, in 64 bits.

Plain numpy from the definitions, one token and one head at a time, sharing no
code with the kernels. Inputs are the stored 16-bit values as float64 (or the
cache as an array of them); results are unrounded.

Bounds. With u the half-spacing of the element type (2^-11 fp16, 2^-8 bf16):

* a turned element a c - b s takes two fp32 products and a sum (3 roundings of
  2^-24) and one rounding to the type:
      |y - ref| <= u |ref| + 2^-22 (|a c| + |b s|) + tiny
  where tiny = 2^-25 is fp16's half-spacing below its normal range (bf16: none
  that matters);
* attention's weights are rounded to the type before they multiply v. With
  A[d] = sum_j w_j |v_jd| (w the exact softmax), S = max_j scale sum_d |q k_j|:
      |y - ref| <= u |ref| + (u + e) A + tiny (1 + sum_j |v_jd|),
      e = 2 D 2^-23 S + (m / 16 + 16) 2^-22 + 2^-20
  for m keys: the scores' fp32 sums, the products' sums (one rounding per 16
  keys, the joins, a factor of two for truncation) and the exponential; tiny
  bounds what the rounding of small weights (relative to a largest one of at
  least 1) and of the result loses below fp16's normal range;
* the logarithm of the sum: |lse - ref| <= e + 2^-22 |ref|.
"""
from __future__ import annotations

import numpy as np

UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -126}


def rope(x, table, positions, pair_axes=None, interleaved=False):
    """x [T, H, D], table [rows, R], positions [axes, T] -> (y, |a c| + |b s|)."""
    x = np.asarray(x, np.float64)
    table = np.asarray(table, np.float64)
    T, H, D = x.shape
    half = table.shape[1] // 2
    y, mag = x.copy(), np.zeros_like(x)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        axis = 0 if pair_axes is None else pair_axes[i]
        for t in range(T):
            c, s = table[positions[axis][t], i], table[positions[axis][t], half + i]
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
            mag[t, :, a] = np.abs(x[t, :, a] * c) + np.abs(x[t, :, b] * s)
            mag[t, :, b] = np.abs(x[t, :, b] * c) + np.abs(x[t, :, a] * s)
    return y, mag


def rope_tolerance(y, mag, dtype):
    return UNIT[dtype] * np.abs(y) + 2.0 ** -22 * mag + TINY[dtype]


def places(q_offsets, kv_lens):
    """Sequence and place of every row (the place is negative where the
    sequence is shorter than its new tokens)."""
    seq, place = [], []
    for b, n in enumerate(kv_lens):
        count = q_offsets[b + 1] - q_offsets[b]
        for i in range(count):
            seq.append(b)
            place.append(n - count + i)
    return np.array(seq, np.int64), np.array(place, np.int64)


def append(cache, rows, page_table, q_offsets, kv_lens):
    """cache [pages, size, G, D] with rows [T, G, D] stored at their places."""
    cache = np.array(cache)
    size = cache.shape[1]
    for t, (b, p) in enumerate(zip(*places(q_offsets, kv_lens))):
        if p >= 0:
            cache[page_table[b][p // size], p % size] = rows[t]
    return cache


def gather(cache, page_table, b, length):
    """The first `length` places of sequence b, in order: [length, G, D]."""
    size = cache.shape[1]
    return np.stack([cache[page_table[b][p // size], p % size] for p in range(length)]) if length else \
        np.zeros((0,) + cache.shape[2:])


def attention(q, k_cache, v_cache, page_table, q_offsets, kv_lens, causal=True, window=0, scale=None):
    """q [T, H, D] -> out [T, H, D], lse [T, H], and what the bounds need:
    A [T, H, D], sum_j |v_jd| [T, H, D], S [T, H], m [T]. Only the places a row
    sees are touched."""
    q = np.asarray(q, np.float64)
    T, H, D = q.shape
    G = k_cache.shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, A, V = np.zeros((T, H, D)), np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, S, m = np.full((T, H), -np.inf), np.zeros((T, H)), np.zeros(T)
    for t, (b, p) in enumerate(zip(*places(q_offsets, kv_lens))):
        end = min(kv_lens[b], p + 1) if causal else kv_lens[b]
        begin = max(0, p - window + 1) if window else 0
        if end <= begin:
            continue
        size = k_cache.shape[1]
        at = [(page_table[b][j // size], j % size) for j in range(begin, end)]
        pages, slots = [i for i, _ in at], [j for _, j in at]
        k, v = k_cache[pages, slots].astype(np.float64), v_cache[pages, slots].astype(np.float64)
        m[t] = end - begin
        for h in range(H):
            g = h // (H // G)
            s = scale * (k[:, g] @ q[t, h])
            top = s.max()
            w = np.exp(s - top)
            total = w.sum()
            lse[t, h] = top + np.log(total)
            w /= total
            out[t, h] = w @ v[:, g]
            A[t, h] = w @ np.abs(v[:, g])
            V[t, h] = np.abs(v[:, g]).sum(0)
            S[t, h] = (scale * (np.abs(k[:, g]) @ np.abs(q[t, h]))).max()
    return out, lse, dict(A=A, V=V, S=S, m=m)


def _slack(D, parts):
    return 2 * D * 2.0 ** -23 * parts["S"] + (parts["m"][:, None] / 16 + 16) * 2.0 ** -22 + 2.0 ** -20


def attention_tolerance(out, parts, dtype):
    u = UNIT[dtype]
    e = _slack(out.shape[2], parts)[..., None]
    return u * np.abs(out) + (u + e) * parts["A"] + TINY[dtype] * (1 + parts["V"])


def lse_tolerance(lse, D, parts):
    with np.errstate(invalid="ignore"):
        return np.where(np.isfinite(lse), _slack(D, parts) + 2.0 ** -22 * np.abs(lse), 0.0)
