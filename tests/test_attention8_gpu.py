"""Attention over an 8-bit paged cache, on the GPU, against the 64-bit oracle
(oracle/attention.py derives the bounds)."""
import ctypes
import time

import numpy as np
import pytest

from oracle import attention as oa
from test_kv_cache8_gpu import FORMS, Rows, _held, _normals, _numbers
from test_paged_attention_canaries_gpu import GUARD, PATTERN, _guarded, _intact
from test_paged_attention_errors_gpu import NORMAL_NS, SHORT_NS, TIMEOUT, _tmem, hooks  # noqa: F401
from test_paged_attention_gpu import DTYPES, HEADS, LENS, Batch, _np, _status_stays_clean, _t, w4  # noqa: F401

pytestmark = pytest.mark.gpu

STEP_ROWS = 48  # past these rows of a cached head the values are rounded to 16 bits


class Batch8(Batch):
    """A batch whose cache is held in 8 bits: scales between 2^-spread and 2^spread of the rows' own, and NaN
    (and bytes that are not zero) in the slots that no place names."""

    def __init__(self, dev, dtype, form, H, G, D, page, lens, seed=0, layout="token", gain=1.0, spread=0.0):
        import torch

        super().__init__(dev, dtype, H, G, D, page, lens, seed=seed, layout="token", poison=None, gain=gain)
        self.form, r = form, torch.Generator().manual_seed(seed + 1)
        pages = self.k.shape[0]
        used = torch.zeros(pages, page, dtype=torch.bool)
        for b, m in enumerate(self.kv):
            for p in range(m):
                used[self.table[b][p // page], p % page] = True
        for name in "kv":
            q, s = oa.hold(_np(getattr(self, name)), form)
            s = torch.from_numpy(s) * 2.0 ** (spread * (2 * torch.rand(s.shape, generator=r) - 1))
            q = torch.from_numpy(q).float().to(_held(form)).view(torch.uint8)
            s[~used], q[~used] = float("nan"), 0x7F  # e4m3: NaN
            s, q = s.float().transpose(1, 2), q
            if layout == "head":
                q = q.transpose(1, 2).contiguous().to(dev).transpose(1, 2)
            elif layout == "joint":  # rows that are wider than a head, scales of k and v side by side
                wide = torch.zeros(pages, page, G, 2 * D, dtype=torch.uint8)
                wide[..., D:] = q
                q = wide.to(dev)[..., D:]
            q = q.to(dev).view(_held(form)) if layout != "joint" else q.view(_held(form))
            scales = torch.zeros(pages, G + 1, 2, page, device=dev)
            scales[:, 1:, 1] = s.to(dev)
            setattr(self, name + "8", q)
            setattr(self, name + "_scale", scales[:, 1:, 1] if layout == "joint" else s.contiguous().to(dev))

    def attend(self, w4, max_q=None, **kw):  # noqa: F811
        return w4.paged_attention(self.q, self.k8, self.v8, self.page_table, self.q_offsets, self.kv_lens,
                                  self.max_q if max_q is None else max_q, k_scale=self.k_scale, v_scale=self.v_scale,
                                  **kw)

    def check(self, out, lse=None, tiles=None, **kw):
        ref, lse_ref, parts = oa.attention8(_np(self.q), _numbers(self.k8), _numbers(self.v8), _np(self.k_scale),
                                            _np(self.v_scale), self.table, self.offsets, self.kv, **kw)
        tiles = self.max_q * self.H // self.G > STEP_ROWS if tiles is None else tiles
        got = _np(out)
        assert np.isfinite(got).all()
        tol = oa.attention8_tolerance(ref, parts, self.dtype, tiles)
        bad = np.abs(got - ref) > tol
        assert not bad.any(), (np.argwhere(bad)[0], (np.abs(got - ref) / tol).max(), int(bad.sum()))
        if lse is not None:
            got = _np(lse)
            empty = np.isneginf(lse_ref)
            assert np.array_equal(np.isneginf(got), empty)
            d = np.abs(np.where(empty, 0, got) - np.where(empty, 0, lse_ref))
            assert (d <= oa.lse8_tolerance(lse_ref, self.D, parts, self.dtype)).all(), d.max()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("H,G,D", HEADS)
def test_attention(w4, cuda_device, H, G, D, lens, form, dtype):  # noqa: F811
    b = Batch8(cuda_device, dtype, form, H, G, D, 16, LENS[lens], seed=H + D)
    b.check(*b.attend(w4, return_lse=True))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("lens", ["one token", "few", "chunks", "short of room", "long"])
@pytest.mark.parametrize("window", [1, 16, 40, 129, 1000, (1 << 31) - 1])
def test_window(w4, cuda_device, lens, window, form):  # noqa: F811
    b = Batch8(cuda_device, "fp16", form, 10, 2, 128, 32, LENS[lens], seed=window % 1000)
    b.check(*b.attend(w4, window=window, return_lse=True), window=window)


@pytest.mark.parametrize("lens", ["one token", "few", "chunks", "empty"])
def test_whole_sequence(w4, cuda_device, lens):  # noqa: F811
    b = Batch8(cuda_device, "bf16", "int8", 14, 2, 64, 16, LENS[lens], seed=3)
    b.check(*b.attend(w4, causal=False, return_lse=True), causal=False)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 112, 128, 256])
@pytest.mark.parametrize("layout", ["token", "head", "joint"])
@pytest.mark.parametrize("lens", ["few", "chunks"])
def test_pages_and_layouts(w4, cuda_device, page, layout, lens):  # noqa: F811
    b = Batch8(cuda_device, "fp16", "int8", 10, 2, 128 if layout == "joint" else 64, page, LENS[lens], seed=page,
               layout=layout)
    b.check(b.attend(w4))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("spread", [3.0, 12.0])
@pytest.mark.parametrize("lens", ["one token", "few", "chunks", "long"])
def test_scales_far_apart(w4, cuda_device, lens, spread, dtype):  # noqa: F811
    """Scales of keys and values that differ by up to 2^24 from place to place."""
    b = Batch8(cuda_device, dtype, "int8", 10, 2, 128, 16, LENS[lens], seed=21, spread=spread, gain=2.0 ** -spread)
    b.check(*b.attend(w4, return_lse=True))


@pytest.mark.parametrize("lens", ["one token", "chunks", "long"])
def test_sharp_scores_and_scale(w4, cuda_device, lens):  # noqa: F811
    b = Batch8(cuda_device, "fp16", "int8", 10, 2, 128, 16, LENS[lens], seed=11, gain=20.0)
    b.check(*b.attend(w4, scale=0.25, return_lse=True), scale=0.25)


@pytest.mark.parametrize("lens", ["one token", "few", "chunks"])
def test_rising_scores(w4, cuda_device, lens):  # noqa: F811
    """Every key scores higher than the one before it, by its scale alone."""
    import torch

    b = Batch8(cuda_device, "fp16", "int8", 10, 2, 128, 16, LENS[lens], seed=12)
    b.k8.fill_(100)
    for s, m in enumerate(b.kv):
        for p in range(m):
            b.k_scale[b.table[s][p // 16], :, p % 16] = 0.0002 * (p + 1)
    b.q.copy_(torch.ones_like(b.q))
    b.check(b.attend(w4))


@pytest.mark.parametrize("lens", [[(1, 700), (1, 40)], [(40, 700), (3, 40)]])
@pytest.mark.parametrize("dtype,k,v", [("fp16", 2.0 ** -20, 2.0 ** -24), ("bf16", 2.0 ** -40, 2.0 ** -50),
                                       ("bf16", 2.0 ** 40, 2.0 ** 45), ("fp16", 500.0, 500.0)])
def test_small_and_large_rows(w4, cuda_device, lens, dtype, k, v):  # noqa: F811
    """Keys and values of other orders than 1: the queries undo the keys' in part."""
    b = Batch8(cuda_device, dtype, "int8", 10, 2, 128, 16, lens, seed=13,
               gain=min(2.0 / k, 10000.0 if dtype == "fp16" else 1e30))
    b.k_scale *= k
    b.v_scale *= v
    if dtype == "fp16":  # what is below its normal range keeps its absolute error only
        assert float(b.q.abs().max()) < 65504
    b.check(*b.attend(w4, return_lse=True))


@pytest.mark.parametrize("q_len", [1, 40])
def test_values_of_zeros(w4, cuda_device, q_len):  # noqa: F811
    """Rows of zeros have the least scale, 2^-100 / 127: whole blocks of them among others, and nothing else."""
    b = Batch8(cuda_device, "bf16", "int8", 10, 2, 64, 16, [(q_len, 700)], seed=14)
    least = 2.0 ** -100 / 127
    for first, last in ((0, 300), (512, 700), (300, 512)):
        for p in range(first, last):
            b.v8[b.table[0][p // 16], p % 16] = 0
            b.v_scale[b.table[0][p // 16], :, p % 16] = least
        b.check(*b.attend(w4, return_lse=True))


@pytest.mark.parametrize("q_len", [1, 3, 40])
def test_a_row_without_numbers_reaches_the_rows_that_see_it(w4, cuda_device, q_len):  # noqa: F811
    """A scale of NaN, of a key or of a value, at a place that every row sees; in another sequence and past the
    length nothing changes."""
    for what in ("k_scale", "v_scale"):
        b = Batch8(cuda_device, "fp16", "int8", 10, 2, 64, 16, [(q_len, 200), (q_len, 90)], seed=15)
        good = b.attend(w4)
        getattr(b, what)[b.table[0][3], 0, 5] = float("nan")
        out = b.attend(w4)
        assert bool(out[:q_len, :5].isnan().all())
        assert bool((out[q_len:] == good[q_len:]).all()) and not bool(out[:q_len, 5:].isnan().any())


def test_pages_before_the_window_are_free(w4, cuda_device):  # noqa: F811
    window, page = 40, 16
    b = Batch8(cuda_device, "fp16", "int8", 10, 2, 128, page, [(1, 300), (3, 200), (130, 500)], seed=16)
    for s, m in enumerate(b.kv):
        n = b.offsets[s + 1] - b.offsets[s]
        for p in range(max(0, m - n - window + 1) // page):
            b.k_scale[b.table[s][p]] = float("nan")
            b.v_scale[b.table[s][p]] = float("nan")
            b.page_table[s, p] = -1
    b.check(b.attend(w4, window=window), window=window)


def test_same_bits_again_and_in_other_batches(w4, cuda_device):  # noqa: F811
    b = Batch8(cuda_device, "fp16", "int8", 10, 2, 128, 16, LENS["long"] + LENS["chunks"], seed=17)
    first = b.attend(w4)
    for _ in range(3):
        assert (b.attend(w4) == first).all()
    b.check(first)
    b.check(b.attend(w4, b.max_q + 500))


def test_many_sequences(w4, cuda_device):  # noqa: F811
    r = np.random.default_rng(18)
    lens = [(int(n), int(n + c)) for n, c in zip(r.integers(0, 3, 700), r.integers(0, 40, 700))]
    b = Batch8(cuda_device, "fp16", "int8", 4, 2, 64, 16, lens, seed=18)
    b.check(b.attend(w4))
    lens = [(int(n), int(n + c)) for n, c in zip(r.integers(0, 40, 300), r.integers(0, 40, 300))]
    b = Batch8(cuda_device, "bf16", "e4m3", 4, 2, 64, 16, lens, seed=19)
    b.check(b.attend(w4))


@pytest.mark.parametrize("q_len", [1, 40])
def test_cache_past_32_bit_offsets(w4, cuda_device, q_len):  # noqa: F811
    """A cache of more than 2^32 bytes, its last pages in use: append, attention, and reading back."""
    import torch

    G, D, page = 8, 128, 64
    pages = (1 << 32) // (page * G * D) + 5
    r = Rows(w4, cuda_device, "fp16", "int8", 16, G, D, page, [(700, 700)], seed=20)
    k, v = (torch.empty(pages, page, G, D, dtype=torch.int8, device=cuda_device) for _ in range(2))
    ks, vs = (torch.empty(pages, G, page, device=cuda_device) for _ in range(2))
    r.append()
    near = r.read(dtype=torch.float16)
    moved = (pages - 1 - r.args[0].clamp(min=0)).contiguous()
    w4.kv_append(r.k, r.v, k, v, moved, *r.args[1:], k_scale=ks, v_scale=vs)
    far = w4.kv_read(k, v, moved, *r.args[1:], 700, dtype=torch.float16, k_scale=ks, v_scale=vs)
    assert all(torch.equal(x, y) for x, y in zip(near, far))
    offsets = torch.tensor([0, q_len], dtype=torch.int32, device=cuda_device)
    q = r.q[:q_len]
    a = w4.paged_attention(q, r.k_cache, r.v_cache, r.args[0], offsets, r.args[2], q_len, k_scale=r.ks, v_scale=r.vs)
    b = w4.paged_attention(q, k, v, moved, offsets, r.args[2], q_len, k_scale=ks, v_scale=vs)
    assert torch.equal(a, b)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("q_lens", [(1, 1, 1), (1, 30, 4)])
def test_graph_of_append_and_attention(w4, cuda_device, q_lens, form):  # noqa: F811
    """The calls together, as a decoder makes them, captured once and replayed as the sequences grow: the
    attention sees what the append stored."""
    import torch

    lens = [(n, n + m) for n, m in zip(q_lens, (100, 30, 241))]
    r = Rows(w4, cuda_device, "fp16", form, 10, 2, 128, 16, [(n, m + 6) for n, m in lens], seed=21)
    first = Rows(w4, cuda_device, "fp16", form, 10, 2, 128, 16, [(m + 6, m + 6) for _, m in lens], seed=22)
    w4.kv_append(first.k, first.v, r.k_cache, r.v_cache, r.args[0], *first.args[1:], k_scale=r.ks, v_scale=r.vs)
    norm = (1 + 0.1 * _normals((128,), 23)).to(cuda_device)
    table = w4.rope_table(400, 128, device=cuda_device)
    qn = torch.empty(r.T, 10, 128, dtype=torch.float16, device=cuda_device)

    def step():
        r.append(q=r.q, table=table, q_norm=norm, k_norm=norm, q_out=qn)
        return w4.paged_attention(qn, r.k_cache, r.v_cache, *r.args, max(q_lens), k_scale=r.ks, v_scale=r.vs)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            out = step()
    for grow in (0, 1, 5):
        kv = [m + grow for _, m in lens]
        r.args[2].copy_(torch.tensor(kv, dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        ref, _, parts = oa.attention8(_np(qn), _numbers(r.k_cache), _numbers(r.v_cache), _np(r.ks), _np(r.vs),
                                      r.table, r.offsets, kv)
        tol = oa.attention8_tolerance(ref, parts, "fp16", max(q_lens) * 5 > STEP_ROWS)
        assert (np.abs(_np(out) - ref) <= tol).all()
        # and the rows are this step's: the last of each is what a 16-bit cache would hold, to 8 bits
        k = oa.head_norm(_np(r.k), _np(norm), np.float32(1e-6))
        _, place = oa.places(r.offsets, kv)
        k, _ = oa.rope(k, _np(table), place[None])
        for b in range(3):
            t, p = r.offsets[b + 1] - 1, kv[b] - 1
            at = r.table[b][p // 16], p % 16
            held = _numbers(r.k_cache)[at] * _np(r.ks)[at[0], :, at[1], None]
            assert (np.abs(held - k[t]) <= oa.held_tolerance(k[t], form, 2.0 ** -19 * np.abs(k[t]).max())[0]).all()


def test_another_stream_and_shared_workspace(w4, cuda_device):  # noqa: F811
    import torch

    b = Batch8(cuda_device, "fp16", "int8", 10, 2, 128, 16, LENS["long"], seed=24)
    c = Batch8(cuda_device, "fp16", "e4m3", 8, 8, 64, 16, LENS["chunks"], seed=25)
    d = Batch(cuda_device, "fp16", 8, 8, 64, 16, LENS["chunks"], seed=26)  # a 16-bit cache in between
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        outs = [b.attend(w4), c.attend(w4), w4.paged_attention(*d.args(), d.max_q), b.attend(w4), c.attend(w4)]
    s.synchronize()
    for x, out in zip((b, c, d, b, c), outs):
        x.check(out)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[(1, 300), (1, 17)], [(3, 900), (1, 1)], [(20, 1500), (25, 25)],
                                  [(130, 400), (1, 9), (51, 3000)]])
def test_attention_writes_only_its_outputs(w4, cuda_device, lens, D, form, dtype):  # noqa: F811
    import torch

    b = Batch8(cuda_device, dtype, form, 10, 2, D, 16, lens, seed=D)
    T = b.offsets[-1]
    buf, out = _guarded((T, 10, D), _t(dtype), cuda_device)
    lse_buf, lse = _guarded((T, 10), torch.float32, cuda_device)
    lib = w4.lib()
    n = int(lib.w4a16_paged_attention_workspace_bytes(T, len(lens), 10, 2, D, b.max_q))
    ws_buf = torch.full((n + 2 * GUARD,), 0x55, dtype=torch.uint8, device=cuda_device)
    ws, st = ws_buf[GUARD:GUARD + n], w4._stream(cuda_device)
    assert lib.w4a16_workspace_init(w4._ptr(ws), n, st) == 0
    c = w4._packed_cache(b.k8, b.v8, b.page_table, b.q_offsets, b.kv_lens, b.q.dtype, 0, b.k8.dtype)[0]
    s = w4._packed_scales(b.k8, b.k_scale, b.v_scale, 0)
    before = [x.view(torch.uint8).clone() for x in (b.k8, b.v8, b.k_scale, b.v_scale, b.fused)]
    for _ in range(2):
        assert lib.w4a16_paged_attention_ex(c, s, T, w4._ptr(b.q), b.q.stride(0), b.q.stride(1), 10, b.max_q, 1, 0,
                                            ctypes.c_float(D ** -0.5), w4._ptr(out), w4._ptr(lse), w4._ptr(ws), n,
                                            st) == 0
    b.check(out, lse)
    assert _intact(buf) and _intact(lse_buf)
    assert bool((ws_buf[:GUARD] == 0x55).all()) and bool((ws_buf[-GUARD:] == 0x55).all())
    for x, y in zip((b.k8, b.v8, b.k_scale, b.v_scale, b.fused), before):
        assert torch.equal(x.view(torch.uint8), y)


@pytest.mark.parametrize("small", [1, 3, 49])
def test_rows_of_a_sequence_longer_than_max_q_len_are_not_written(w4, cuda_device, small):  # noqa: F811
    import torch

    b = Batch8(cuda_device, "fp16", "int8", 10, 2, 128, 16, [(50, 100), (1, 40), (1, 300)], seed=27)
    out = torch.full((52, 10, 128), 7.0, dtype=torch.float16, device=cuda_device)
    b.attend(w4, small, out=out)
    assert w4.device_status(raise_on_error=False) == 6
    assert bool((out[:50] == 7.0).all())
    good = b.attend(w4, 50)
    b.check(good)
    out[:50] = good[:50]
    b.check(out)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("G,H", [(2, 10), (8, 40)])
def test_append_and_read_write_only_their_outputs(w4, cuda_device, G, H, form):  # noqa: F811
    """Caches, scales, q_out and the rows read between guards; a cache whose heads are part of a wider row."""
    import torch

    r = Rows(w4, cuda_device, "fp16", form, H, G, 64, 16, [(1, 20), (9, 40), (70, 70)], seed=H)
    pages, T = r.k_cache.shape[0], r.T
    bufs, wide = zip(*[_guarded((pages, 16, G + 1, 64), torch.int16, cuda_device) for _ in range(2)])
    wide = [x.view(torch.uint8).view(pages, 16, G + 1, 128) for x in wide]
    k, v = (x[:, :, :G, :64].view(_held(form)) for x in wide)
    s_bufs, scales = zip(*[_guarded((pages, G + 1, 16), torch.float32, cuda_device) for _ in range(2)])
    ks, vs = (x[:, :G] for x in scales)
    q_buf, q_out = _guarded((T, H, 64), torch.float16, cuda_device)
    r.append()
    q = w4.kv_append(r.k, r.v, k, v, *r.args, q=r.q, q_out=q_out, k_scale=ks, v_scale=vs)
    assert q is q_out and torch.equal(q_out, r.q)
    assert all(_intact(x) for x in (*bufs, *s_bufs, q_buf))
    mark = torch.full((1,), PATTERN, dtype=torch.int16, device=cuda_device).view(torch.uint8)
    for x, s, cache, scale in ((wide[0], scales[0], r.k_cache, r.ks), (wide[1], scales[1], r.v_cache, r.vs)):
        rest = x[:, :, :G, 64:].reshape(-1, 2), x[:, :, G].reshape(-1, 2)
        assert all(bool((y == mark).all()) for y in rest)
        assert bool((s[:, G].view(torch.int32) == PATTERN).all())
        held, was = x[:, :, :G, :64], cache.view(torch.uint8)
        stored = (scale != 0).transpose(1, 2)
        assert torch.equal(held[stored], was[stored])
        assert bool((held[~stored].reshape(-1, 2) == mark).all())
    bufs, rows = zip(*[_guarded((T, G, 64), torch.float16, cuda_device) for _ in range(2)])
    w4.kv_read(k, v, *r.args, T, k_out=rows[0], v_out=rows[1], k_scale=ks, v_scale=vs)
    assert all(_intact(x) for x in bufs)
    assert all(torch.equal(x, y) for x, y in zip(rows, r.read(dtype=torch.float16)))


def test_append_from_16_bit_views_of_another_shape_is_refused(w4, cuda_device):  # noqa: F811
    import torch

    r = Rows(w4, cuda_device, "fp16", "int8", 4, 2, 64, 16, [(2, 20)])
    with pytest.raises(ValueError):
        w4.kv_append(r.k, r.v, r.k_cache, r.v_cache, *r.args)                     # no scales
    with pytest.raises(ValueError):
        w4.kv_append(r.k, r.v, r.k_cache, r.v_cache.view(torch.float8_e4m3fn), *r.args, k_scale=r.ks, v_scale=r.vs)
    with pytest.raises(ValueError):
        w4.kv_append(r.k, r.v, r.k_cache, r.v_cache, *r.args, k_scale=r.ks.cpu(), v_scale=r.vs)
    with pytest.raises(ValueError):
        w4.kv_append(r.k, r.v, r.k_cache, r.v_cache, *r.args, k_scale=r.ks, v_scale=r.vs,
                     q_norm=torch.ones(64, device=cuda_device))                   # without q
    with pytest.raises(ValueError):
        r.read()                                                                  # no dtype
    with pytest.raises(ValueError):
        r.read(dtype=torch.float32)
    with pytest.raises(ValueError):
        w4.paged_attention(r.q, r.k_cache, r.v_cache, *r.args, 2)
    with pytest.raises(w4.W4A16Error):
        narrow = r.k_cache.reshape(-1)[8:-56].view(torch.int8)  # a base that is not on 16 bytes
        narrow = narrow[:narrow.numel() // (16 * 2 * 64) * (16 * 2 * 64)].view(-1, 16, 2, 64)
        w4.kv_read(narrow, narrow, *r.args, 2, dtype=torch.float16, k_scale=r.ks[:len(narrow)],
                   v_scale=r.vs[:len(narrow)])


# ------------------------------------------------------- bounded waits of the tiles --

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,limits", [([(300, 4000)], (0, 1, 2, 3)), ([(20, 30000)], (0, 1, 2, 3)),
                                         ([(200, 200), (100, 700)], (0, 1))])
def test_wait_times_out_and_next_call_is_correct(hooks, cuda_device, lens, limits, D):  # noqa: F811
    """As for 16-bit caches: converters that stop after a few blocks, and a 1 ms limit."""
    import torch

    import w4a16_group_quantized_linear_gb300 as w4

    lib = hooks
    b = Batch8(cuda_device, "bf16", "int8", 10, 2, D, 16, lens, seed=40)
    T = b.offsets[-1]
    c = w4._packed_cache(b.k8, b.v8, b.page_table, b.q_offsets, b.kv_lens, b.q.dtype, 0, b.k8.dtype)[0]
    s = w4._packed_scales(b.k8, b.k_scale, b.v_scale, 0)
    out = torch.empty(T, 10, D, dtype=torch.bfloat16, device=cuda_device)
    n = int(lib.w4a16_paged_attention_workspace_bytes(T, len(lens), 10, 2, D, b.max_q))
    ws = torch.empty(n, dtype=torch.uint8, device=cuda_device)
    st = w4._stream(cuda_device)

    def call():
        assert lib.w4a16_workspace_init(w4._ptr(ws), n, st) == 0
        return lib.w4a16_paged_attention_ex(c, s, T, w4._ptr(b.q), b.q.stride(0), b.q.stride(1), 10, b.max_q, 1, 0,
                                            D ** -0.5, w4._ptr(out), None, w4._ptr(ws), n, st)

    for issue_limit in limits:
        a0, f0 = _tmem(lib)
        assert lib.w4a16_test_set_hooks(SHORT_NS, issue_limit) == 0
        assert call() == 0
        t0 = time.perf_counter()
        assert lib.w4a16_device_status(st) == TIMEOUT, issue_limit
        assert time.perf_counter() - t0 < 1.0
        a1, f1 = _tmem(lib)
        assert a1 - a0 > 0 and a1 - a0 == f1 - f0
    assert lib.w4a16_test_set_hooks(NORMAL_NS, -1) == 0
    assert call() == 0
    assert lib.w4a16_device_status(st) == 0
    b.check(out)


# ------------------------------------------------------------- many cached heads --

@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("H,G,q_len", [(12, 12, 1), (100, 100, 2), (613, 613, 1), (330, 330, 1), (26, 13, 3)])
def test_head_counts_that_do_not_divide_the_thread_blocks(w4, cuda_device, H, G, q_len, form):  # noqa: F811
    """Single tokens work on many cached heads side by side, in several turns where there are more of them than
    thread blocks or a rest would be idle: every head of every sequence, the last turn's missing ones among them."""
    b = Batch8(cuda_device, "fp16", form, H, G, 64, 16, [(q_len, 200), (q_len, 17), (q_len, 130)], seed=H)
    b.check(*b.attend(w4, return_lse=True))


def test_caches_that_were_never_appended_to(w4, cuda_device):  # noqa: F811
    """Scales of 0, as of a cache made with torch.zeros, count as rows of zeros: among others, and alone."""
    for q_len in (1, 40):
        b = Batch8(cuda_device, "fp16", "int8", 10, 2, 64, 16, [(q_len, 300)], seed=30)
        for first, last in ((64, 200), (0, 300)):
            for p in range(first, last):
                at = b.table[0][p // 16], slice(None), p % 16
                b.k_scale[at] = 0
                b.v_scale[at] = 0
            b.check(*b.attend(w4, return_lse=True))


@pytest.mark.parametrize("cache", FORMS)
@pytest.mark.parametrize("steps", [1, 5])
def test_example(cuda_device, steps, cache):
    """The decoder example over an 8-bit cache: chunks and single tokens see the same rows. Their kernels' outputs
    differ by the roundings of the bounds above, of values that the two quantized projections leave near 1."""
    import importlib.util
    import os

    from conftest import ROOT

    spec = importlib.util.spec_from_file_location("decoder_attention",
                                                  os.path.join(ROOT, "examples", "decoder_attention.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    grown, whole = example.run(steps=steps, cache=cache)
    assert grown.shape == whole.shape and bool(grown.isfinite().all())
    assert float((grown.float() - whole.float()).abs().max()) <= 0.01 * float(whole.float().abs().max())
