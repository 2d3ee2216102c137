"""Cases for the 8-bit paged cache of the serving path: norms of the query and
key heads with the position rotation in the same pass, keys and values stored
in 8 bits with a scale for each row as they are appended, rows read back in 16
bits, and attention of new tokens over such a cache.

Every case is a dict of plain values. ``prepare`` builds what a serving
program holds before the call (the fused projection's output, the norms'
weights, the cache with its scales, the page table and the lengths, all on the
GPU); ``run`` makes one pass, with the framework's calls when ``own`` is set
and with elementary torch operations in 32 bits otherwise; ``exact`` is the
definition in 64 bits.

A row x of a cached head is held as integers q in [-127, 127] or as e4m3
numbers q, and one fp32 scale: s = max(max|x|, 2^-100) / 127 (or 448), q = x / s
rounded to nearest. It stands for q s.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
CACHES = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}  # type, its largest value
DEVICE = "cuda:0"
TABLE_ROWS = 1 << 18  # positions the rotary table covers
ROTARY_BASE = 1.0e6
EPS = 1e-6
LEAST = 2.0 ** -100  # what a row's largest value is taken for if it is less


# ------------------------------------------------------------------- cases --

def listed():
    """40 query and 8 key/value heads of 128 are the heads of a 5120-wide layer
    (the width of the repository's decode shapes); the 64-wide heads are a
    generic small layout."""
    big = dict(heads=40, kv_heads=8, dim=128)
    small = dict(heads=32, kv_heads=4, dim=64)
    return [
        # the queries of one image of 26 x 46 patches in an encoder that normalises heads, rotated by (time,
        # height, width)
        dict(name="norm_image", op="rope", dtype="fp16", tokens=1196, heads=48, dim=128, rotary=128, axes=3,
             pattern="blocks", interleaved=False),
        # 20 frames of video, half of each head rotated, adjacent elements paired
        dict(name="norm_video", op="rope", dtype="bf16", tokens=15360, heads=18, dim=128, rotary=64, axes=3,
             pattern="cycle", interleaved=True),
        # a single user's next token: latency alone
        dict(name="append_step_1", op="append", dtype="fp16", cache="e4m3", **big, rotary=128, axes=1,
             pattern="blocks", interleaved=False, page=16, batch=1, singles=1, q_min=1, q_max=1, ctx_min=1024,
             ctx_max=1024, lens=1),
        # a decode batch of 89 sequences with 7 short chunks in it, three axes; what was stored is read back, as for
        # another worker
        dict(name="append_batch", op="append", dtype="bf16", cache="int8", **small, rotary=32, axes=3,
             pattern="blocks", interleaved=True, page=48, batch=96, singles=89, q_min=9, q_max=130, ctx_min=20,
             ctx_max=700, lens=2),
        # a few prompts prefilled together
        dict(name="append_prompts", op="append", dtype="fp16", cache="e4m3", **big, rotary=128, axes=1,
             pattern="blocks", interleaved=False, page=64, batch=4, singles=0, q_min=900, q_max=3500, ctx_min=0,
             ctx_max=0, lens=3),
        # a shared prefix of a long document handed to a worker that keeps 16 bits
        dict(name="read_prefix", op="read", dtype="fp16", cache="int8", **big, page=64, batch=1, singles=0,
             q_min=30011, q_max=30011, ctx_min=0, ctx_max=0, lens=4),
        # the last few places of many short sequences
        dict(name="read_ragged", op="read", dtype="bf16", cache="e4m3", **small, page=16, batch=50, singles=11,
             q_min=3, q_max=77, ctx_min=0, ctx_max=900, lens=5),
        # a single user's next token after a short conversation: latency alone
        dict(name="attn_step_1", op="attention", dtype="fp16", cache="int8", **big, page=16, batch=1, singles=1,
             q_min=1, q_max=1, ctx_min=776, ctx_max=776, window=0, causal=True, lse=False, lens=6),
        # a full decode batch of ragged lengths: the cache's bytes count
        dict(name="attn_step_64", op="attention", dtype="fp16", cache="int8", **big, page=16, batch=64, singles=64,
             q_min=1, q_max=1, ctx_min=300, ctx_max=8000, window=0, causal=True, lse=False, lens=7),
        # two very long documents being answered: one token each, the cache split over the whole GPU
        dict(name="attn_step_long", op="attention", dtype="bf16", cache="e4m3", **big, page=64, batch=2, singles=2,
             q_min=1, q_max=1, ctx_min=120001, ctx_max=150001, window=0, causal=True, lse=True, lens=8),
        # a chunk of a long prompt over what is already in the cache: the tensor cores count
        dict(name="attn_chunk", op="attention", dtype="fp16", cache="int8", **big, page=64, batch=1, singles=0,
             q_min=2048, q_max=2048, ctx_min=28000, ctx_max=28000, window=0, causal=True, lse=False, lens=9),
        # decode rows and prompt chunks in one batch, sliding window
        dict(name="attn_mixed_window", op="attention", dtype="bf16", cache="int8", **small, page=16, batch=14,
             singles=8, q_min=257, q_max=2000, ctx_min=500, ctx_max=4000, window=1024, causal=True, lse=True,
             lens=10),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads, kv_heads, dim = rng.choice([(40, 8, 128), (16, 2, 128), (32, 4, 64), (14, 2, 64), (8, 8, 128),
                                       (12, 12, 64), (32, 2, 128), (20, 1, 64)])
    base = dict(dtype=rng.choice(["fp16", "bf16"]), lens=rng.randrange(100, 1 << 30))
    op = rng.choice(["rope", "append", "append", "read", "attention", "attention", "attention", "attention"])
    turn = dict(rotary=rng.choice([dim, dim, dim // 2]), axes=rng.choice([1, 2, 3]),
                pattern=rng.choice(["blocks", "cycle"]), interleaved=rng.random() < 0.5)
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "rope":
        most = min(16384, 30_000_000 // (heads * dim))
        return dict(op=op, dtype=base["dtype"], tokens=_log_int(rng, 1, most), heads=heads, dim=dim, **turn)
    base.update(cache=rng.choice(["int8", "e4m3"]), heads=heads, kv_heads=kv_heads, dim=dim, page=page)
    if op in ("append", "read"):
        rest = dict(turn) if op == "append" else {}
        if rng.random() < 0.5:
            batch = _log_int(rng, 1, 128)
            return dict(op=op, **base, **rest, batch=batch, singles=batch, q_min=1, q_max=1, ctx_min=0,
                        ctx_max=_log_int(rng, 16, 700))
        batch = rng.randint(1, 6)
        most = _log_int(rng, 40, 2200)
        return dict(op=op, **base, **rest, batch=batch, singles=rng.randint(0, batch - 1), q_min=max(2, most // 3),
                    q_max=most, ctx_min=0, ctx_max=_log_int(rng, 16, 700))
    rest = dict(window=rng.choice([0, 0, 100, 777, 4096]), causal=True, lse=rng.random() < 0.5)
    kind = rng.choice(["step", "step", "verify", "chunk", "mixed"])
    if kind in ("step", "verify"):
        batch = _log_int(rng, 1, 64)
        q = 1 if kind == "step" else rng.randint(2, 9)
        # all cached tokens together stay below those of the two long documents
        ctx = _log_int(rng, 64, min(120000, 200000 // (batch * kv_heads * dim // 1024 + 1)) if batch > 1 else 120000)
        return dict(op=op, **base, batch=batch, singles=batch if q == 1 else 0, q_min=q, q_max=q,
                    ctx_min=max(1, ctx // 8), ctx_max=ctx, **rest)
    if kind == "chunk":
        q = _log_int(rng, 33, 2000)
        ctx = _log_int(rng, 1, 24000)
        if ctx < 2000 and rng.random() < 0.3:
            rest.update(causal=False, window=0)
        return dict(op=op, **base, batch=1, singles=0, q_min=q, q_max=q, ctx_min=ctx, ctx_max=ctx, **rest)
    batch = rng.randint(2, 12)
    return dict(op=op, **base, batch=batch, singles=rng.randint(1, batch - 1), q_min=20,
                q_max=_log_int(rng, 40, 1500), ctx_min=0, ctx_max=_log_int(rng, 64, 4000), **rest)


def _lengths(case):
    """New tokens and cached-plus-new tokens of each sequence, in batch order."""
    r = random.Random(case["lens"])
    q = [1] * case["singles"] + [r.randint(case["q_min"], case["q_max"])
                                 for _ in range(case["batch"] - case["singles"])]
    r.shuffle(q)
    return q, [n + r.randint(case["ctx_min"], case["ctx_max"]) for n in q]


def _pair_axes(case):
    """Which axis turns each of the rotary / 2 pairs."""
    half, axes = case["rotary"] // 2, case["axes"]
    if case["pattern"] == "cycle":
        return [i % axes for i in range(half)]
    return [min(axes - 1, i * axes // half) for i in range(half)]


def work(case):
    if case["op"] == "rope":
        x = case["tokens"] * case["heads"] * case["dim"]
        turned = case["tokens"] * case["heads"] * case["rotary"]
        return {"bytes": 4 * x + 4 * case["tokens"] * (case["axes"] + case["rotary"]) + 4 * case["dim"],
                "flops": 4 * x + 3 * turned}
    q_lens, kv_lens = _lengths(case)
    T, H, G, D = sum(q_lens), case["heads"], case["kv_heads"], case["dim"]
    held = 2 * T * G * (D + 4)    # the rows' keys and values, and their scales, as the cache holds them
    rows = 2 * 2 * T * G * D      # the same in 16 bits
    if case["op"] == "read":
        return {"bytes": held + rows, "flops": 2 * T * G * D}
    if case["op"] == "append":
        # q, k and v are read, q is written, and k and v in the cache; one table row per token
        moved = 4 * T * H * D + rows + held + 4 * T * (case["axes"] + case["rotary"]) + 8 * D
        return {"bytes": moved + (held + rows if case["cache"] == "int8" else 0),
                "flops": 4 * T * (H + G) * D + 3 * T * (H + G) * case["rotary"] + 6 * T * G * D}
    seen, pairs = 0, 0
    for n, m in zip(q_lens, kv_lens):
        first = max(0, m - n - case["window"] + 1) if case["window"] else 0
        seen += m - first
        if not case["causal"]:
            pairs += n * m
        elif case["window"]:
            pairs += sum(min(m - n + i + 1, case["window"]) for i in range(n))
        else:
            pairs += n * (m - n) + n * (n + 1) // 2
    return {"bytes": 4 * T * H * D + 2 * seen * G * (D + 4) + (4 * T * H if case["lse"] else 0),
            "flops": 4 * pairs * H * D}


# ------------------------------------------------------------------ inputs --

def _table(rotary):
    """cos and sin of every position: fp32 [TABLE_ROWS, rotary]."""
    inv = ROTARY_BASE ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=DEVICE) / rotary)
    a = torch.arange(TABLE_ROWS, dtype=torch.float64, device=DEVICE)[:, None] * inv[None, :]
    return torch.cat((a.cos(), a.sin()), dim=1).float()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEVICE)


def _quantise(x, cache):
    """x [..., D] in 32 bits -> (values of the cache's type, scale [...])."""
    dtype, most = CACHES[cache]
    top = x.abs().amax(-1).clamp(min=LEAST)
    y = x * (torch.full_like(top, most) / top)[..., None]
    return y.round().to(dtype) if dtype == torch.int8 else y.to(dtype), top / most


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32)

    st = dict(case)
    D = case["dim"]
    if case["op"] in ("rope", "append"):
        st["table"] = _table(case["rotary"])
        st["pair_axes"], st["pair_index"] = _pair_axes(case), _ints(_pair_axes(case)).long()
        st["q_norm"], st["k_norm"] = 1 + 0.2 * normal(D), 1 + 0.2 * normal(D)
    if case["op"] == "rope":
        T, H = case["tokens"], case["heads"]
        # the query and key part of a projection's rows, which also hold the values
        fused = (3 * normal(T, (H + max(1, H // 8)) * D)).to(dt)
        st["x"] = fused[:, :H * D].unflatten(1, (H, D))
        t = torch.arange(T, device=DEVICE)
        start = int(torch.randint(0, 4000, (1,), generator=gen, device=DEVICE))
        rows = [start + t // 768, start + t // 46, start + t % 46]  # frame, row and column of a patch
        st["positions"] = torch.stack(rows[:case["axes"]] if case["axes"] > 1 else [start + t]).to(torch.int32)
        return st

    q_lens, kv_lens = _lengths(case)
    T, H, G, page = sum(q_lens), case["heads"], case["kv_heads"], case["page"]
    need = [-(-m // page) for m in kv_lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.full((len(need), max(max(need), 1)), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    offsets = [0]
    for n in q_lens:
        offsets.append(offsets[-1] + n)
    st.update(page_table=table, q_offsets=_ints(offsets), kv_lens=_ints(kv_lens), max_q_len=max(q_lens), rows=T,
              longest=max(kv_lens))
    # a few elements of a head's keys are larger than the rest, and rows differ in size
    channel = torch.where(torch.arange(D, device=DEVICE) % 16 == 5, 3.0, 1.0)
    channel = channel / channel.square().mean().sqrt()
    for name, by in (("k", channel), ("v", torch.ones(D, device=DEVICE))):
        x = normal(pages, page, G, D) * by * torch.exp(0.2 * normal(pages, page, G, 1))
        st[name + "_cache"], scale = _quantise(x, case["cache"])
        st[name + "_scale"] = scale.transpose(1, 2).contiguous()  # [pages, kv_heads, page]
        del x
    if case["op"] == "append":
        fused = (2 * normal(T, (H + 2 * G) * D)).to(dt)
        st["q"] = fused[:, :H * D].unflatten(1, (H, D))
        st["k"] = fused[:, H * D:(H + G) * D].unflatten(1, (G, D))
        st["v"] = fused[:, (H + G) * D:].unflatten(1, (G, D))
        st["positions"] = None  # the place in the sequence
        if case["axes"] > 1:
            st["positions"] = torch.randint(0, 5000, (case["axes"], T), generator=gen, device=DEVICE,
                                            dtype=torch.int32)
    elif case["op"] == "attention":
        # heads differ in how sharply they look: logits with a spread of 0.5 to 3
        gain = 0.5 + 2.5 * torch.rand(1, H, 1, generator=gen, device=DEVICE)
        st["q"] = (normal(T, H, D) * gain).to(dt)
    return st


# --------------------------------------------------------------- one pass --

def run(state):
    return {"rope": _rope, "append": _append, "read": _read, "attention": _attention}[state["op"]](state)


def _normalise(x, weight):
    """x [..., D] in 32 bits, divided by its root mean square and multiplied by the weight."""
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


def _turn(x, cos, sin, interleaved):
    """x [T, heads, dim] in 32 bits; cos, sin [T, pairs]."""
    n = 2 * cos.shape[1]
    c, s = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    else:
        a, b = x[..., :n // 2], x[..., n // 2:n]
        turned = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    return torch.cat((turned, x[..., n:]), dim=-1)


def _angles(table, positions, pair_index):
    """cos, sin [T, pairs]: each pair takes the position of its axis. positions [axes, T]."""
    half = table.shape[1] // 2
    at = positions.long()[pair_index]   # [pairs, T]
    pair = torch.arange(half, device=positions.device)[:, None]
    return table[at, pair].T, table[at, pair + half].T


def _rope(st):
    if own:
        import w4a16_group_quantized_linear_gb300 as w4
        return w4.rope(st["x"], st["positions"], st["table"], pair_axes=st["pair_axes"],
                       interleaved=st["interleaved"], norm=st["q_norm"], eps=EPS)
    cos, sin = _angles(st["table"], st["positions"], st["pair_index"])
    return _turn(_normalise(st["x"].float(), st["q_norm"]), cos, sin, st["interleaved"]).to(st["x"].dtype)


def _places(st):
    """Sequence and place of every row of the call, and the page and slot that hold it."""
    t = torch.arange(st["rows"], device=DEVICE)
    offsets = st["q_offsets"].long()
    b = torch.searchsorted(offsets[1:], t, right=True)
    place = st["kv_lens"].long()[b] - offsets[b + 1] + t
    return b, place, st["page_table"].long()[b, place // st["page"]], place % st["page"]


def _read(st):
    if own:
        import w4a16_group_quantized_linear_gb300 as w4
        return w4.kv_read(st["k_cache"], st["v_cache"], st["page_table"], st["q_offsets"], st["kv_lens"], st["rows"],
                          dtype=DTYPES[st["dtype"]], k_scale=st["k_scale"], v_scale=st["v_scale"])
    _, _, page, slot = _places(st)

    def rows(cache, scale):
        held = cache.view(torch.uint8)[page, slot].view(cache.dtype).float()
        return (held * scale[page, :, slot][..., None]).to(DTYPES[st["dtype"]])

    return rows(st["k_cache"], st["k_scale"]), rows(st["v_cache"], st["v_scale"])


def _append(st):
    caches = st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"]
    if own:
        import w4a16_group_quantized_linear_gb300 as w4
        q = w4.kv_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["page_table"], st["q_offsets"],
                         st["kv_lens"], q=st["q"], table=st["table"], positions=st["positions"],
                         pair_axes=st["pair_axes"], interleaved=st["interleaved"], q_norm=st["q_norm"],
                         k_norm=st["k_norm"], eps=EPS, k_scale=st["k_scale"], v_scale=st["v_scale"])
    else:
        _, place, page, slot = _places(st)
        positions = st["positions"] if st["positions"] is not None else place[None]
        cos, sin = _angles(st["table"], positions, st["pair_index"])
        k = _turn(_normalise(st["k"].float(), st["k_norm"]), cos, sin, st["interleaved"])
        for x, cache, scale in ((k, *caches[0::2]), (st["v"].float(), *caches[1::2])):
            held, of = _quantise(x, st["cache"])
            cache.view(torch.uint8)[page, slot] = held.view(torch.uint8)
            scale[page, :, slot] = of
        q = _turn(_normalise(st["q"].float(), st["q_norm"]), cos, sin, st["interleaved"]).to(st["q"].dtype)
    # integers come back as the values they stand for
    return (q, *_read(st)) if st["cache"] == "int8" else (q, *caches)


def _attention(st):
    if own:
        import w4a16_group_quantized_linear_gb300 as w4
        return w4.paged_attention(st["q"], st["k_cache"], st["v_cache"], st["page_table"], st["q_offsets"],
                                  st["kv_lens"], st["max_q_len"], causal=st["causal"], window=st["window"],
                                  return_lse=st["lse"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    H, G, D = st["heads"], st["kv_heads"], st["dim"]
    B, n, m = st["batch"], st["max_q_len"], st["longest"]
    pages = st["page_table"][:, :-(-m // st["page"])].long().clamp(min=0)

    def values(cache, scale):  # [B, G, places, D]
        held = cache.view(torch.uint8)[pages].view(cache.dtype).float() * scale[pages].transpose(-1, -2)[..., None]
        return held.flatten(1, 2)[:, :m].transpose(1, 2)

    # every sequence's rows, as many as the longest has: [B, G, heads that share it * n, D]
    offsets, length = st["q_offsets"].long(), st["kv_lens"].long()
    i = torch.arange(n, device=DEVICE)
    count = offsets[1:] - offsets[:-1]
    rows = (offsets[:-1, None] + i).clamp(max=st["rows"] - 1)
    q = st["q"][rows].float().view(B, n, G, H // G, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
    scores = torch.matmul(q, values(st["k_cache"], st["k_scale"]).transpose(-1, -2)).view(B, G, H // G, n, m)
    scores *= D ** -0.5
    place = (length - count)[:, None] + i
    at = torch.arange(m, device=DEVICE)
    hidden = at >= length[:, None, None]
    if st["causal"]:
        hidden = hidden | (at > place[..., None])
    if st["window"]:
        hidden = hidden | (at <= place[..., None] - st["window"])
    scores.masked_fill_(hidden[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), values(st["v_cache"], st["v_scale"])).view(B, G, H // G, n, D) / total
    t = torch.arange(st["rows"], device=DEVICE)
    b = torch.searchsorted(offsets[1:], t, right=True)
    mine = b, t - offsets[b]
    out = out.permute(0, 3, 1, 2, 4)[mine].flatten(1, 2).to(st["q"].dtype)
    if not st["lse"]:
        return out
    return out, (top + torch.log(total))[..., 0].permute(0, 3, 1, 2)[mine].flatten(1, 2)


# ------------------------------------------------------------------- exact --

def _head_exact(x, weight, table, positions, pair_axes, interleaved):
    """A head divided by its norm, weighted, and its pairs multiplied as complex numbers, in 64 bits."""
    half = table.shape[1] // 2
    x = x.double()
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    for i in range(half):
        row = table.double()[positions[pair_axes[i]].long()]
        w = torch.complex(row[:, i], row[:, half + i])[:, None]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        z = torch.complex(x[..., a], x[..., b]) * w
        x[..., a], x[..., b] = z.real, z.imag
    return x


def _held_exact(x, cache):
    """(q, scale) of rows in 64 bits: integers, or the nearest numbers of 3 fraction bits from 2^-6 to 448 and of
    multiples of 2^-9 below."""
    most = CACHES[cache][1]
    scale = x.abs().max(-1).values.clamp(min=LEAST) / most
    y = x / scale[..., None]
    if cache == "int8":
        return torch.round(y), scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-most, most), scale


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _head_exact(st["x"], st["q_norm"], st["table"], st["positions"], st["pair_axes"], case["interleaved"])
    q_lens, kv_lens = _lengths(case)
    page, H, G, D = case["page"], case["heads"], case["kv_heads"], case["dim"]
    slots = [st["page_table"][b].long().repeat_interleave(page)[:m] * page
             + torch.arange(m, device=DEVICE) % page for b, m in enumerate(kv_lens)]
    new = torch.cat([s[m - n:] for s, n, m in zip(slots, q_lens, kv_lens)])
    scales = [st[name].double().transpose(1, 2).reshape(-1, G) for name in ("k_scale", "v_scale")]
    if case["op"] == "read":
        return tuple(st[name].view(-1, G, D).view(torch.uint8)[new].view(st[name].dtype).double() * s[new][..., None]
                     for name, s in zip(("k_cache", "v_cache"), scales))
    if case["op"] == "append":
        positions = st["positions"]
        if positions is None:
            positions = torch.cat([torch.arange(m - n, m, device=DEVICE) for n, m in zip(q_lens, kv_lens)])[None]
        how = (st["table"], positions, st["pair_axes"], case["interleaved"])
        k = _held_exact(_head_exact(st["k"], st["k_norm"], *how), case["cache"])
        v = _held_exact(st["v"].double(), case["cache"])
        q = _head_exact(st["q"], st["q_norm"], *how)
        if case["cache"] == "int8":
            return q, k[0] * k[1][..., None], v[0] * v[1][..., None]
        caches = [st[name].double() for name in ("k_cache", "v_cache")]
        for i, held in enumerate((k, v)):
            caches[i].view(-1, G, D)[new] = held[0]
            scales[i][new] = held[1]
        return q, *caches, *(s.view(-1, page, G).transpose(1, 2).contiguous() for s in scales)
    T = sum(q_lens)
    out = torch.empty(T, H, D, dtype=torch.float64, device=DEVICE)
    lse = torch.empty(T, H, dtype=torch.float64, device=DEVICE)
    t0 = 0
    for n, m, s in zip(q_lens, kv_lens, slots):
        i = torch.arange(m - n, m, device=DEVICE)[:, None]
        j = torch.arange(m, device=DEVICE)[None, :]
        unseen = torch.zeros(n, m, dtype=torch.bool, device=DEVICE)
        if case["causal"]:
            unseen |= j > i
        if case["window"]:
            unseen |= j <= i - case["window"]
        for g in range(G):
            k, v = (st[name].view(-1, G, D)[:, g].view(torch.uint8)[s].view(st[name].dtype).double()
                    * scales[x][s, g, None] for x, name in enumerate(("k_cache", "v_cache")))
            for h in range(g * (H // G), (g + 1) * (H // G)):
                a = st["q"][t0:t0 + n, h].double() @ k.T / math.sqrt(D)
                a[unseen] = -math.inf
                lse[t0:t0 + n, h] = torch.logsumexp(a, dim=1)
                out[t0:t0 + n, h] = torch.softmax(a, dim=1) @ v
        t0 += n
    return (out, lse) if case["lse"] else out
