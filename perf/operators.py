"""Cases for the attention operators of the serving path: rotary positions
(one or several axes), appending keys and values to a paged cache with the
rotation applied on the way, and attention of new tokens over that cache.

Every case is a dict of plain values. ``prepare`` builds what a serving
program holds before the call (the fused projection's output, the paged cache,
the page table and the lengths, all on the GPU); ``run`` makes one pass, with
the framework's calls when ``own`` is set and with elementary torch operations
in 32 bits otherwise; ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
DEVICE = "cuda:0"
TABLE_ROWS = 1 << 18  # positions the rotary table covers
ROTARY_BASE = 1.0e6


# ------------------------------------------------------------------- cases --

def listed():
    """40 query and 8 key/value heads of 128 are the heads of a 5120-wide layer
    (the width of the repository's decode shapes), 16 and 2 those of its
    2048-wide one; the 64-wide heads are a generic small layout."""
    big = dict(heads=40, kv_heads=8, dim=128)
    small = dict(heads=32, kv_heads=4, dim=64)
    return [
        # one image of 26 x 46 patches entering a prompt, rotated by (time, height, width)
        dict(name="rope_image", op="rope", dtype="fp16", tokens=1196, heads=48, dim=128, rotary=128, axes=3,
             pattern="blocks", interleaved=False),
        # 20 frames of video, the axes dealt out to the pairs in turn, adjacent elements paired
        dict(name="rope_video", op="rope", dtype="bf16", tokens=15360, heads=18, dim=128, rotary=128, axes=3,
             pattern="cycle", interleaved=True),
        # a single user's next token: latency alone
        dict(name="append_step_1", op="append", dtype="fp16", **big, rotary=128, axes=1, pattern="blocks",
             interleaved=False, page=16, batch=1, singles=1, q_min=1, q_max=1, ctx_min=1024, ctx_max=1024, lens=1),
        # a decode batch: one token of each of 96 sequences
        dict(name="append_step_96", op="append", dtype="fp16", **big, rotary=128, axes=1, pattern="blocks",
             interleaved=False, page=16, batch=96, singles=96, q_min=1, q_max=1, ctx_min=20, ctx_max=700, lens=2),
        # a few prompts prefilled together
        dict(name="append_prompts", op="append", dtype="fp16", **big, rotary=128, axes=1, pattern="blocks",
             interleaved=False, page=64, batch=4, singles=0, q_min=900, q_max=3500, ctx_min=0, ctx_max=0, lens=3),
        # small heads with a partly rotated width, three axes and single-token rows among prompt chunks
        dict(name="append_axes", op="append", dtype="bf16", **small, rotary=32, axes=3, pattern="blocks",
             interleaved=True, page=48, batch=9, singles=5, q_min=301, q_max=1500, ctx_min=0, ctx_max=600, lens=4),
        # a single user's next token after a short conversation: latency alone
        dict(name="attn_step_1", op="attention", dtype="fp16", **big, page=16, batch=1, singles=1, q_min=1, q_max=1,
             ctx_min=776, ctx_max=776, window=0, causal=True, lse=False, lens=5),
        # a full decode batch of ragged lengths: the cache's bytes count
        dict(name="attn_step_64", op="attention", dtype="fp16", **big, page=16, batch=64, singles=64, q_min=1,
             q_max=1, ctx_min=300, ctx_max=8000, window=0, causal=True, lse=False, lens=6),
        # two very long documents being answered: one token each, the cache split over the whole GPU
        dict(name="attn_step_long", op="attention", dtype="bf16", **big, page=64, batch=2, singles=2, q_min=1,
             q_max=1, ctx_min=120001, ctx_max=150001, window=0, causal=True, lse=True, lens=7),
        # draft tokens being verified: a few rows of each of 16 sequences
        dict(name="attn_verify", op="attention", dtype="fp16", **big, page=32, batch=16, singles=0, q_min=5, q_max=5,
             ctx_min=2000, ctx_max=9000, window=0, causal=True, lse=False, lens=8),
        # a chunk of a long prompt over what is already in the cache: the tensor cores count
        dict(name="attn_chunk", op="attention", dtype="fp16", **big, page=64, batch=1, singles=0, q_min=2048,
             q_max=2048, ctx_min=28000, ctx_max=28000, window=0, causal=True, lse=False, lens=9),
        # decode rows and prompt chunks in one batch, sliding window
        dict(name="attn_mixed_window", op="attention", dtype="bf16", **small, page=16, batch=14, singles=8,
             q_min=257, q_max=2000, ctx_min=500, ctx_max=4000, window=1024, causal=True, lse=True, lens=10),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads, kv_heads, dim = rng.choice([(40, 8, 128), (16, 2, 128), (32, 4, 64), (14, 2, 64), (8, 8, 128),
                                       (12, 12, 64), (32, 2, 128), (20, 1, 64)])
    layout = dict(heads=heads, kv_heads=kv_heads, dim=dim)
    dtype = rng.choice(["fp16", "bf16"])
    lens = rng.randrange(100, 1 << 30)
    op = rng.choice(["rope", "append", "append", "attention", "attention", "attention"])
    rotary = rng.choice([dim, dim, dim // 2])
    turn = dict(rotary=rotary, axes=rng.choice([1, 2, 3]), pattern=rng.choice(["blocks", "cycle"]),
                interleaved=rng.random() < 0.5)
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "rope":
        most = min(16384, 30_000_000 // (heads * dim))
        return dict(op=op, dtype=dtype, tokens=_log_int(rng, 1, most), heads=heads, dim=dim, **turn)
    if op == "append":
        if rng.random() < 0.5:
            batch = _log_int(rng, 1, 128)
            return dict(op=op, dtype=dtype, **layout, **turn, page=page, batch=batch, singles=batch, q_min=1, q_max=1,
                        ctx_min=0, ctx_max=_log_int(rng, 16, 700), lens=lens)
        batch = rng.randint(1, 6)
        most = _log_int(rng, 40, 2200)
        return dict(op=op, dtype=dtype, **layout, **turn, page=page, batch=batch, singles=rng.randint(0, batch - 1),
                    q_min=max(2, most // 3), q_max=most, ctx_min=0, ctx_max=_log_int(rng, 16, 700), lens=lens)
    rest = dict(window=rng.choice([0, 0, 100, 777, 4096]), causal=True, lse=rng.random() < 0.5, lens=lens)
    kind = rng.choice(["step", "step", "verify", "chunk", "mixed"])
    if kind in ("step", "verify"):
        batch = _log_int(rng, 1, 64)
        q = 1 if kind == "step" else rng.randint(2, 9)
        # all cached tokens together stay below those of the two long documents
        ctx = _log_int(rng, 64, min(120000, 200000 // (batch * kv_heads * dim // 1024 + 1)) if batch > 1 else 120000)
        return dict(op=op, dtype=dtype, **layout, page=page, batch=batch, singles=batch if q == 1 else 0, q_min=q,
                    q_max=q, ctx_min=max(1, ctx // 8), ctx_max=ctx, **rest)
    if kind == "chunk":
        q = _log_int(rng, 33, 2000)
        ctx = _log_int(rng, 1, 24000)
        if ctx < 2000 and rng.random() < 0.3:
            rest.update(causal=False, window=0)
        return dict(op=op, dtype=dtype, **layout, page=page, batch=1, singles=0, q_min=q, q_max=q, ctx_min=ctx,
                    ctx_max=ctx, **rest)
    batch = rng.randint(2, 12)
    return dict(op=op, dtype=dtype, **layout, page=page, batch=batch, singles=rng.randint(1, batch - 1),
                q_min=20, q_max=_log_int(rng, 40, 1500), ctx_min=0, ctx_max=_log_int(rng, 64, 4000), **rest)


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
    size = 2
    if case["op"] == "rope":
        x = case["tokens"] * case["heads"] * case["dim"]
        turned = case["tokens"] * case["heads"] * case["rotary"]
        return {"bytes": 2 * size * x + 4 * case["tokens"] * (case["axes"] + case["rotary"]), "flops": 3 * turned}
    q_lens, kv_lens = _lengths(case)
    T, H, G, D = sum(q_lens), case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        # q, k and v are read; q, and k and v in the cache, are written; one table row per token
        return {"bytes": 2 * size * T * (H + 2 * G) * D + 4 * T * (case["axes"] + case["rotary"]),
                "flops": 3 * T * (H + G) * case["rotary"]}
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
    return {"bytes": 2 * size * T * H * D + 2 * size * seen * G * D + (4 * T * H if case["lse"] else 0),
            "flops": 4 * pairs * H * D}


# ------------------------------------------------------------------ inputs --

def _table(rotary):
    """cos and sin of every position: fp32 [TABLE_ROWS, rotary]."""
    inv = ROTARY_BASE ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=DEVICE) / rotary)
    a = torch.arange(TABLE_ROWS, dtype=torch.float64, device=DEVICE)[:, None] * inv[None, :]
    return torch.cat((a.cos(), a.sin()), dim=1).float()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEVICE)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32).to(dt)

    st = dict(case)
    if case["op"] == "rope":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        # the query and key part of a projection's rows, which also hold the values
        fused = normal(T, (H + max(1, H // 8)) * D)
        st["x"] = fused[:, :H * D].unflatten(1, (H, D))
        st["table"] = _table(case["rotary"])
        t = torch.arange(T, device=DEVICE)
        start = int(torch.randint(0, 4000, (1,), generator=gen, device=DEVICE))
        rows = [start + t // 768, start + t // 46, start + t % 46]  # frame, row and column of a patch
        st["positions"] = torch.stack(rows[:case["axes"]] if case["axes"] > 1 else [start + t]).to(torch.int32)
        st["pair_axes"], st["pair_index"] = _pair_axes(case), _ints(_pair_axes(case)).long()
        return st

    q_lens, kv_lens = _lengths(case)
    T, H, G, D, page = sum(q_lens), case["heads"], case["kv_heads"], case["dim"], case["page"]
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
    st.update(page_table=table, q_offsets=_ints(offsets), kv_lens=_ints(kv_lens), max_q_len=max(q_lens),
              k_cache=normal(pages, page, G, D), v_cache=normal(pages, page, G, D))
    if case["op"] == "append":
        fused = normal(T, (H + 2 * G) * D)
        st["q"] = fused[:, :H * D].unflatten(1, (H, D))
        st["k"] = fused[:, H * D:(H + G) * D].unflatten(1, (G, D))
        st["v"] = fused[:, (H + G) * D:].unflatten(1, (G, D))
        st["table"] = _table(case["rotary"])
        st["pair_axes"], st["pair_index"] = _pair_axes(case), _ints(_pair_axes(case)).long()
        st["positions"] = None  # the place in the sequence
        if case["axes"] > 1:
            st["positions"] = torch.randint(0, 5000, (case["axes"], T), generator=gen, device=DEVICE,
                                            dtype=torch.int32)
    else:
        # heads differ in how sharply they look: logits with a spread of 0.5 to 3
        gain = 0.5 + 2.5 * torch.rand(1, H, 1, generator=gen, device=DEVICE)
        st["q"] = (torch.randn(T, H, D, generator=gen, device=DEVICE) * gain).to(dt)
        # the list form of the lengths, which the program that forms the batch has anyway
        st["q_lens"], st["kv_list"] = q_lens, kv_lens
    return st


# --------------------------------------------------------------- one pass --

def run(state):
    return {"rope": _rope, "append": _append, "attention": _attention}[state["op"]](state)


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
                       interleaved=st["interleaved"])
    cos, sin = _angles(st["table"], st["positions"], st["pair_index"])
    return _turn(st["x"].float(), cos, sin, st["interleaved"]).to(st["x"].dtype)


def _append(st):
    if own:
        import w4a16_group_quantized_linear_gb300 as w4
        q = w4.kv_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["page_table"], st["q_offsets"],
                         st["kv_lens"], q=st["q"], table=st["table"], positions=st["positions"],
                         pair_axes=st["pair_axes"], interleaved=st["interleaved"])
        return q, st["k_cache"], st["v_cache"]
    T, page, dt = st["q"].shape[0], st["page"], st["q"].dtype
    t = torch.arange(T, device=DEVICE)
    offsets = st["q_offsets"].long()
    b = torch.searchsorted(offsets[1:], t, right=True)
    place = st["kv_lens"].long()[b] - offsets[b + 1] + t
    positions = st["positions"] if st["positions"] is not None else place[None]
    cos, sin = _angles(st["table"], positions, st["pair_index"])
    slot = st["page_table"].long()[b, place // page], place % page
    st["k_cache"][slot] = _turn(st["k"].float(), cos, sin, st["interleaved"]).to(dt)
    st["v_cache"][slot] = st["v"]
    return _turn(st["q"].float(), cos, sin, st["interleaved"]).to(dt), st["k_cache"], st["v_cache"]


def _softmax_sums(q, k, v, place, length, window, causal):
    """q [..., G, r, n, D], k and v [..., G, m, D], place [..., n] and length [...] of each
    sequence; returns out [..., G, r, n, D] and the logarithm of the sum [..., G, r, n]."""
    m = k.shape[-2]
    scores = torch.matmul(q, k.unsqueeze(-3).transpose(-1, -2)) * (q.shape[-1] ** -0.5)
    at = torch.arange(m, device=DEVICE)
    seen = (at < length[..., None]).unsqueeze(-2)
    if causal:
        seen = seen & (at <= place[..., None])
    if window:
        seen = seen & (at > place[..., None] - window)
    scores = scores.masked_fill(~seen[..., None, None, :, :], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v.unsqueeze(-3)) / total, (top + torch.log(total))[..., 0]


def _attention(st):
    if own:
        import w4a16_group_quantized_linear_gb300 as w4
        return w4.paged_attention(st["q"], st["k_cache"], st["v_cache"], st["page_table"], st["q_offsets"],
                                  st["kv_lens"], st["max_q_len"], causal=st["causal"], window=st["window"],
                                  return_lse=st["lse"])
    H, G, D, page = st["heads"], st["kv_heads"], st["dim"], st["page"]
    q_lens, kv_lens = st["q_lens"], st["kv_list"]

    def keys(cache, pages):  # [..., m, G, D] in 32 bits, then heads first
        return cache[pages.long().clamp(min=0)].flatten(-4, -3).float().transpose(-3, -2)

    def some(first, count):
        """`count` consecutive sequences of equally many new tokens, at once."""
        n = q_lens[first]
        t0 = sum(q_lens[:first])
        longest = max(kv_lens[first:first + count])
        pages = st["page_table"][first:first + count, :-(-longest // page)]
        q = st["q"][t0:t0 + count * n].float().view(count, n, G, H // G, D).permute(0, 2, 3, 1, 4)
        length = st["kv_lens"][first:first + count].long()
        place = length[:, None] - n + torch.arange(n, device=DEVICE)
        out, lse = _softmax_sums(q, keys(st["k_cache"], pages), keys(st["v_cache"], pages), place, length,
                                 st["window"], st["causal"])
        return (out.permute(0, 3, 1, 2, 4).reshape(count * n, H, D).to(st["q"].dtype),
                lse.permute(0, 3, 1, 2).reshape(count * n, H))

    if min(q_lens) == max(q_lens):
        parts = [some(0, len(q_lens))]
    else:
        parts = [some(b, 1) for b in range(len(q_lens))]
    out = torch.cat([o for o, _ in parts])
    return (out, torch.cat([s for _, s in parts])) if st["lse"] else out


# ------------------------------------------------------------------- exact --

def _turn_exact(x, table, positions, pair_axes, interleaved):
    """The rotation as a product of complex numbers in 64 bits."""
    half = table.shape[1] // 2
    x = x.double().clone()
    for i in range(half):
        row = table.double()[positions[pair_axes[i]].long()]
        w = torch.complex(row[:, i], row[:, half + i])[:, None]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        z = torch.complex(x[..., a], x[..., b]) * w
        x[..., a], x[..., b] = z.real, z.imag
    return x


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _turn_exact(st["x"], st["table"], st["positions"], st["pair_axes"], case["interleaved"])
    q_lens, kv_lens = _lengths(case)
    page, H, G, D = case["page"], case["heads"], case["kv_heads"], case["dim"]
    slots = [st["page_table"][b].long().repeat_interleave(page)[:m] * page
             + torch.arange(m, device=DEVICE) % page for b, m in enumerate(kv_lens)]
    if case["op"] == "append":
        positions = st["positions"]
        if positions is None:
            positions = torch.cat([torch.arange(m - n, m, device=DEVICE) for n, m in zip(q_lens, kv_lens)])[None]
        where = torch.cat([s[m - n:] for s, n, m in zip(slots, q_lens, kv_lens)])
        how = (st["table"], positions, st["pair_axes"], case["interleaved"])
        k, v = st["k_cache"].double(), st["v_cache"].double()
        k.view(-1, G, D)[where] = _turn_exact(st["k"], *how)
        v.view(-1, G, D)[where] = st["v"].double()
        return _turn_exact(st["q"], *how), k, v
    T = sum(q_lens)
    out = torch.empty(T, H, D, dtype=torch.float64, device=DEVICE)
    lse = torch.empty(T, H, dtype=torch.float64, device=DEVICE)
    t0 = 0
    for n, m, s in zip(q_lens, kv_lens, slots):
        i = torch.arange(m - n, m, device=DEVICE)[:, None]
        j = torch.arange(m, device=DEVICE)[None, :]
        hidden = torch.zeros(n, m, dtype=torch.bool, device=DEVICE)
        if case["causal"]:
            hidden |= j > i
        if case["window"]:
            hidden |= j <= i - case["window"]
        for h in range(H):
            g = h // (H // G)
            k = st["k_cache"].view(-1, G, D)[s, g].double()
            v = st["v_cache"].view(-1, G, D)[s, g].double()
            a = st["q"][t0:t0 + n, h].double() @ k.T / math.sqrt(D)
            a[hidden] = -math.inf
            lse[t0:t0 + n, h] = torch.logsumexp(a, dim=1)
            out[t0:t0 + n, h] = torch.softmax(a, dim=1) @ v
        t0 += n
    return (out, lse) if case["lse"] else out
