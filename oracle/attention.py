"""Rotary positions, head norms, the paged cache in 16 and 8 bits and attention
over it, in 64 bits.

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

* a head's norm x / sqrt(mean x^2 + eps) w: the mean takes at most 22 fp32 roundings
  (16 elements in a row, 5 sums over threads, the division), eps one; the
  reciprocal root halves them and adds 2 ulp; two products follow. In all n = 20
  2^-24 of the value, on top of what turns it:
      |y - ref| <= u |ref| + n |ref| + (2^-22 + n) (|a c| + |b s|) + tiny
* a row in 8 bits: x / s is off by two roundings of 2^-24 before it goes to the
  nearest integer (at most 127 of them: 2^-16 of a step) or the nearest e4m3
  number (half a step is 2^-4 of the value, or 2^-10 of s below its normal range):
      |q s - ref| <= (1/2 + 2^-15) s + d,  or  max(2^-4 |ref|, 2^-10 s) (1 + 2^-10) + d
  where d is how far the row itself may be off, and |s - ref| <= (d + 2^-22 max|x|) / most;
* attention over 8-bit rows: the integers are exact in the products and the
  weights p_j s_j (s_j the value's scale) are rounded to the type, so the bounds
  are those of the 16-bit cache, but for small weights, which are relative to
  a largest weight times scale: fp16's tiny (1 + max_j s_j sum_j |q_jd|), as the
  products run in fp16 whatever the type. bf16 queries go to fp16 divided by a power
  of two of the row's largest element m_q: exact above 2^-14 of it, else off by 2^-25
  of it, a score by r = 2^-24 scale m_q max_j sum_d |k_jd|, and a weight by twice that
  (it and the sum):
      |y - ref| <= u |ref| + (w + e + 2 r) A + ...,   |lse - ref| <= ... + r
  with w = 2^-11, the rounding of the weights. In whole tiles their factor is that of 32 places, which some of the
  rows may not see, so tiny takes 2 s_v sum_j |q_jd|, s_v the sequence's largest scale. There the bound
  has room besides for values that are rounded to fp16 as q s, each off by w of itself or by twice 2^-25 in
  fp16's own units, of which 2^6 at least make the largest scale: w A + 2^-30 s_v.
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


NORM = 20 * 2.0 ** -24

MOST = {"int8": 127.0, "e4m3": 448.0}
LEAST = 2.0 ** -100  # what a row's largest element is taken for if it is less


def head_norm(x, weight, eps):
    """x [..., D] / sqrt(mean(x^2) + eps) * weight."""
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def norm_rope_tolerance(y, mag, dtype):
    return (UNIT[dtype] + NORM) * np.abs(y) + (2.0 ** -22 + NORM) * mag + TINY[dtype]


def e4m3(x):
    """The nearest e4m3 number (ties to even), held to 448."""
    x = np.asarray(x, np.float64)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def hold(x, form):
    """Rows x [..., D] in 8 bits: (q, scale [...])."""
    x = np.asarray(x, np.float64)
    scale = np.maximum(np.abs(x).max(-1), LEAST) / MOST[form]
    y = x / scale[..., None]
    return np.rint(y) if form == "int8" else e4m3(y), scale


def held_tolerance(x, form, off=0.0):
    """How far q s may be from the row x [..., D], and s from its scale; off: what the row itself may be off."""
    top = np.maximum(np.abs(x).max(-1), LEAST)
    worst = np.max(np.broadcast_to(off, x.shape), -1)
    scale = (top + worst) / MOST[form] * (1 + 2.0 ** -22)
    s = scale[..., None]
    step = (0.5 + 2.0 ** -15) * s if form == "int8" else \
        np.maximum(2.0 ** -4 * (np.abs(x) + off), 2.0 ** -10 * s) * (1 + 2.0 ** -10)
    return step + off, (worst + 2.0 ** -22 * top) / MOST[form]


def attention8(q, k, v, k_scale, v_scale, page_table, q_offsets, kv_lens, **kw):
    """attention() over the rows that an 8-bit cache holds: k, v [pages, size, G, D] the values as held,
    k_scale, v_scale [pages, G, size]. parts["V"] is what bounds the small weights there."""
    def rows(x, s):
        return np.asarray(x, np.float64) * np.swapaxes(np.asarray(s, np.float64), 1, 2)[..., None]

    out, lse, parts = attention(q, rows(k, k_scale), rows(v, v_scale), page_table, q_offsets, kv_lens, **kw)
    T, H, D = out.shape
    G, size = k.shape[2], k.shape[1]
    causal, window = kw.get("causal", True), kw.get("window", 0)
    scale = D ** -0.5 if kw.get("scale") is None else kw["scale"]
    q = np.abs(np.asarray(q, np.float64))
    parts.update(V=np.zeros((T, H, D)), all_V=np.zeros((T, H, D)), Q=np.zeros((T, H)), s_v=np.zeros((T, H)))
    for t, (b, p) in enumerate(zip(*places(q_offsets, kv_lens))):
        end = min(kv_lens[b], p + 1) if causal else kv_lens[b]
        at = range(max(0, p - window + 1) if window else 0, end)
        if not len(at):
            continue
        pages, slots = [page_table[b][j // size] for j in at], [j % size for j in at]
        begin = max(0, kv_lens[b] - (q_offsets[b + 1] - q_offsets[b]) - window + 1) if window else 0
        live = [(page_table[b][j // size], j % size) for j in range(begin, kv_lens[b])]  # what some row sees
        for g in range(G):
            mine = slice(g * (H // G), (g + 1) * (H // G))
            ks, vs = (np.asarray(s, np.float64) for s in (k_scale, v_scale))
            held = np.abs(np.asarray(v, np.float64)[pages, slots, g]).sum(0)
            keys = np.abs(np.asarray(k, np.float64)[pages, slots, g]).sum(1) * ks[pages, g, slots]
            s_v = np.nanmax([vs[i, g, j] for i, j in live])
            parts["V"][t, mine] = vs[pages, g, slots].max() * held
            parts["all_V"][t, mine] = 2 * s_v * held
            parts["Q"][t, mine] = 2.0 ** -24 * scale * q[t, mine].max(-1) * keys.max()
            parts["s_v"][t, mine] = s_v
    return out, lse, parts


def attention8_tolerance(out, parts, dtype, rounded=False):
    """rounded: whole tiles, with room for values that are brought to fp16 as q s first."""
    u, w = UNIT[dtype], UNIT["fp16"]
    r = parts["Q"] if dtype == "bf16" else 0.0
    e = (_slack(out.shape[2], parts) + 2 * r + (w if rounded else 0.0))[..., None]
    tol = u * np.abs(out) + (w + e) * parts["A"] + TINY["fp16"] * (1 + parts["all_V" if rounded else "V"])
    return tol + (2.0 ** -30 * parts["s_v"][..., None] if rounded else 0.0)


def lse8_tolerance(lse, D, parts, dtype):
    return lse_tolerance(lse, D, parts) + np.where(np.isfinite(lse), parts["Q"] if dtype == "bf16" else 0.0, 0.0)
