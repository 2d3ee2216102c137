"""Rotary positions, the paged cache and attention over it, on the GPU, against
the 64-bit oracle (oracle/attention.py derives the bounds)."""
import ctypes

import numpy as np
import pytest

from oracle import attention as oa

pytestmark = pytest.mark.gpu

DTYPES = ["fp16", "bf16"]


@pytest.fixture(scope="module")
def w4():
    import w4a16_group_quantized_linear_gb300 as w4

    w4.lib()
    return w4


@pytest.fixture(autouse=True)
def _status_stays_clean(w4, cuda_device):
    yield
    assert w4.device_status(raise_on_error=False) == 0


def _t(dtype):
    import torch

    return {"fp16": torch.float16, "bf16": torch.bfloat16}[dtype]


def _np(t):
    return t.double().cpu().numpy()


class Batch:
    """A paged cache with every slot that no place names poisoned, and page
    table entries past a sequence's end left invalid."""

    def __init__(self, dev, dtype, H, G, D, page, lens, seed=0, layout="token", poison=float("nan"), gain=1.0):
        import torch

        g = torch.Generator(device="cpu").manual_seed(seed)
        dt = _t(dtype)
        q_lens, self.kv = [n for n, _ in lens], [m for _, m in lens]
        need = [-(-m // page) for m in self.kv]
        pages = sum(need) + 2
        width = max(need + [1]) + 1
        order = torch.randperm(pages, generator=g).tolist()
        self.table = [[-1 - 7 * b] * width for b in range(len(lens))]
        at = 0
        for b, n in enumerate(need):
            self.table[b][:n] = order[at:at + n]
            at += n
        self.offsets = np.concatenate([[0], np.cumsum(q_lens)]).astype(int).tolist()
        T = self.offsets[-1]
        shape = {"token": (pages, page, G, D), "head": (pages, G, page, D), "joint": (pages, 2, page, G, D)}[layout]
        self.D, self.G, self.H, self.page, self.dtype = D, G, H, page, dtype

        def values(shape):
            return torch.randn(*shape, generator=g).to(dt)

        if layout == "joint":
            both = values(shape).to(dev)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = values(shape).to(dev), values(shape).to(dev)
            if layout == "head":
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        used = torch.zeros(pages, page, dtype=torch.bool)
        for b, m in enumerate(self.kv):
            for p in range(m):
                used[self.table[b][p // page], p % page] = True
        if poison is not None:
            self.k[~used.to(dev)] = poison
            self.v[~used.to(dev)] = poison
        # q as a strided part of a fused row
        self.fused = (gain * torch.randn(T, (H + 2) * D, generator=g)).to(dt).to(dev)
        self.q = self.fused[:, D:(H + 1) * D].unflatten(1, (H, D))
        i32 = dict(dtype=torch.int32, device=dev)
        self.page_table, self.q_offsets = torch.tensor(self.table, **i32), torch.tensor(self.offsets, **i32)
        self.kv_lens = torch.tensor(self.kv, **i32)
        self.max_q = max(q_lens)

    def args(self):
        return self.q, self.k, self.v, self.page_table, self.q_offsets, self.kv_lens

    def check(self, out, lse=None, **kw):
        ref, lse_ref, parts = oa.attention(_np(self.q), _np(self.k), _np(self.v), self.table, self.offsets, self.kv,
                                           **kw)
        got = _np(out)
        assert np.isfinite(got).all()
        tol = oa.attention_tolerance(ref, parts, self.dtype)
        bad = np.abs(got - ref) > tol
        assert not bad.any(), (np.argwhere(bad)[0], (np.abs(got - ref) / tol).max(), int(bad.sum()))
        if lse is not None:
            got = _np(lse)
            empty = np.isneginf(lse_ref)
            assert np.array_equal(np.isneginf(got), empty)
            d = np.abs(np.where(empty, 0, got) - np.where(empty, 0, lse_ref))
            assert (d <= oa.lse_tolerance(lse_ref, self.D, parts)).all(), d.max()


HEADS = [(5, 1, 128), (8, 8, 64), (14, 2, 64), (32, 2, 128), (20, 1, 64), (10, 2, 128), (1, 1, 128)]
LENS = {
    "one token": [(1, 1), (1, 15), (1, 16), (1, 17), (1, 300), (1, 64), (1, 129)],
    "empty": [(1, 0), (1, 5), (0, 40), (0, 0), (1, 33)],
    "few": [(3, 3), (5, 130), (0, 40), (2, 64), (4, 257)],
    "short of room": [(7, 4), (2, 40), (3, 0), (1, 128)],
    "chunks": [(130, 130), (57, 300), (1, 129), (64, 513)],
    "one chunk": [(97, 1000)],
    "long": [(1, 3001), (2, 1500)],
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("H,G,D", HEADS)
def test_attention(w4, cuda_device, H, G, D, lens, dtype):
    b = Batch(cuda_device, dtype, H, G, D, 16, LENS[lens], seed=H + D)
    out, lse = w4.paged_attention(*b.args(), b.max_q, return_lse=True)
    b.check(out, lse)


@pytest.mark.parametrize("lens", ["one token", "few", "chunks", "short of room", "long"])
@pytest.mark.parametrize("window", [1, 16, 40, 129, 1000])
def test_window(w4, cuda_device, lens, window):
    b = Batch(cuda_device, "fp16", 10, 2, 128, 32, LENS[lens], seed=window)
    out, lse = w4.paged_attention(*b.args(), b.max_q, window=window, return_lse=True)
    b.check(out, lse, window=window)


@pytest.mark.parametrize("lens", ["one token", "few", "chunks", "empty"])
def test_whole_sequence(w4, cuda_device, lens):
    b = Batch(cuda_device, "bf16", 14, 2, 64, 16, LENS[lens], seed=3)
    out, lse = w4.paged_attention(*b.args(), b.max_q, causal=False, return_lse=True)
    b.check(out, lse, causal=False)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 112, 128, 256])
@pytest.mark.parametrize("layout", ["token", "head", "joint"])
@pytest.mark.parametrize("lens", ["few", "chunks"])
def test_pages_and_layouts(w4, cuda_device, page, layout, lens):
    b = Batch(cuda_device, "fp16", 10, 2, 128 if layout == "joint" else 64, page, LENS[lens], seed=page,
              layout=layout)
    b.check(w4.paged_attention(*b.args(), b.max_q))


@pytest.mark.parametrize("lens", ["one token", "chunks", "long"])
def test_sharp_scores_and_scale(w4, cuda_device, lens):
    """Scores with a spread of tens: the running maximum moves often."""
    b = Batch(cuda_device, "fp16", 10, 2, 128, 16, LENS[lens], seed=11, gain=20.0)
    out, lse = w4.paged_attention(*b.args(), b.max_q, scale=0.25, return_lse=True)
    b.check(out, lse, scale=0.25)


@pytest.mark.parametrize("lens", ["one token", "few", "chunks"])
def test_rising_scores(w4, cuda_device, lens):
    """Every key scores higher than the one before it: each tile raises the maximum by far."""
    import torch

    b = Batch(cuda_device, "fp16", 10, 2, 128, 16, LENS[lens], seed=12)
    for s, m in enumerate(b.kv):
        for p in range(m):
            b.k[b.table[s][p // 16], p % 16] = 0.02 * p
    b.q.copy_(torch.ones_like(b.q))
    b.check(w4.paged_attention(*b.args(), b.max_q))


def test_infinite_stale_slots(w4, cuda_device):
    for lens in ("one token", "chunks"):
        b = Batch(cuda_device, "fp16", 10, 2, 128, 16, LENS[lens], seed=13, poison=float("inf"))
        b.check(w4.paged_attention(*b.args(), b.max_q))


def test_pages_before_the_window_are_free(w4, cuda_device):
    """Pages that no row sees any more may be given away: their entries and what
    they hold are never used."""
    window, page = 40, 16
    b = Batch(cuda_device, "fp16", 10, 2, 128, page, [(1, 300), (3, 200), (130, 500)], seed=14)
    for s, m in enumerate(b.kv):
        n = b.offsets[s + 1] - b.offsets[s]
        for p in range(max(0, m - n - window + 1) // page):
            b.k[b.table[s][p]] = float("nan")
            b.v[b.table[s][p]] = float("nan")
            b.page_table[s, p] = -1
    b.check(w4.paged_attention(*b.args(), b.max_q, window=window), window=window)


def test_same_bits_again_and_in_other_batches(w4, cuda_device):
    b = Batch(cuda_device, "fp16", 10, 2, 128, 16, LENS["long"] + LENS["chunks"], seed=15)
    first = w4.paged_attention(*b.args(), b.max_q)
    for _ in range(3):
        assert (w4.paged_attention(*b.args(), b.max_q) == first).all()
    # a larger max_q_len only chooses kernels
    b.check(w4.paged_attention(*b.args(), b.max_q + 500))


def test_many_sequences(w4, cuda_device):
    r = np.random.default_rng(16)
    lens = [(int(n), int(n + c)) for n, c in zip(r.integers(0, 3, 700), r.integers(0, 40, 700))]
    b = Batch(cuda_device, "fp16", 4, 2, 64, 16, lens, seed=16)
    b.check(w4.paged_attention(*b.args(), b.max_q))
    lens = [(int(n), int(n + c)) for n, c in zip(r.integers(0, 40, 300), r.integers(0, 40, 300))]
    b = Batch(cuda_device, "fp16", 4, 2, 64, 16, lens, seed=17)
    b.check(w4.paged_attention(*b.args(), b.max_q))


@pytest.mark.parametrize("q_len", [1, 40])
def test_cache_past_32_bit_offsets(w4, cuda_device, q_len):
    """A cache of more than 2^32 bytes, its last pages in use."""
    import torch

    G, D, page = 8, 128, 64
    pages = (1 << 32) // (page * G * D) + 5   # > 2^32 elements in each of k and v
    small = Batch(cuda_device, "fp16", 16, G, D, page, [(q_len, 700)], seed=18)
    k = torch.empty(pages, page, G, D, dtype=torch.float16, device=cuda_device)
    v = torch.empty_like(k)
    moved = pages - 1 - small.page_table.clamp(min=0)
    for p in range(11):
        k[moved[0, p]], v[moved[0, p]] = small.k[small.page_table[0, p]], small.v[small.page_table[0, p]]
    out = w4.paged_attention(small.q, k, v, moved, small.q_offsets, small.kv_lens, q_len)
    small.check(out)
    # and the append reaches them
    kn = torch.randn(q_len, G, D, device=cuda_device).half()
    w4.kv_append(kn, kn, k, v, moved, small.q_offsets, small.kv_lens)
    for i in range(q_len):
        p = 700 - q_len + i
        assert (k[moved[0, p // page], p % page] == kn[i]).all() and (v[moved[0, p // page], p % page] == kn[i]).all()


def test_graph_follows_the_lengths(w4, cuda_device):
    """One captured decode step, replayed as the sequences grow."""
    import torch

    lens = [(1, 100), (1, 30), (1, 241)]
    b = Batch(cuda_device, "fp16", 10, 2, 128, 16, [(1, m + 6) for _, m in lens], seed=19, poison=0.5)
    table = w4.rope_table(400, 128, device=cuda_device)
    kn, vn = (torch.randn(3, 2, 128, device=cuda_device).half() for _ in range(2))
    qn, out = torch.empty(3, 10, 128, dtype=torch.float16, device=cuda_device), None

    def step():
        w4.kv_append(kn, vn, b.k, b.v, b.page_table, b.q_offsets, b.kv_lens, q=b.q, table=table, q_out=qn)
        return w4.paged_attention(qn, *b.args()[1:], 1)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            out = step()
    for grow in (0, 1, 5):
        b.kv = [m + grow for _, m in lens]
        b.kv_lens.copy_(torch.tensor(b.kv, dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        q = b.q
        b.q = qn
        b.check(out)
        b.q = q


def test_another_stream_and_shared_workspace(w4, cuda_device):
    import torch

    b = Batch(cuda_device, "fp16", 10, 2, 128, 16, LENS["long"], seed=20)
    c = Batch(cuda_device, "fp16", 8, 8, 64, 16, LENS["chunks"], seed=21)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        outs = [w4.paged_attention(*x.args(), x.max_q) for x in (b, c, b, c)]
    s.synchronize()
    for x, out in zip((b, c, b, c), outs):
        x.check(out)


# ------------------------------------------------------------ rope, append --

def _positions(r, axes, T, rows):
    return r.integers(0, rows, (axes, T)).astype(np.int32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes,pattern", [(1, None), (3, "blocks"), (3, "cycle"), (4, "cycle")])
@pytest.mark.parametrize("T,H,D,R", [(1, 5, 128, 128), (7, 3, 64, 32), (33, 1, 80, 80), (130, 9, 256, 256),
                                     (2500, 22, 64, 64)])
def test_rope(w4, cuda_device, T, H, D, R, axes, pattern, interleaved, dtype):
    import torch

    r = np.random.default_rng(T + H)
    x = torch.from_numpy(r.normal(size=(T, H + 2, D))).to(_t(dtype)).to(cuda_device)[:, 1:H + 1]
    table = w4.rope_table(5000, R, base=1e5, device=cuda_device)
    pos = _positions(r, axes, T, 5000)
    half = R // 2
    pa = None if pattern is None else [i % axes if pattern == "cycle" else i * axes // half for i in range(half)]
    y = w4.rope(x, torch.from_numpy(pos).to(cuda_device), table, pair_axes=pa, interleaved=interleaved)
    rows = slice(0, T) if T < 200 else slice(T - 40, T)
    ref, mag = oa.rope(_np(x)[rows], _np(table), pos[:, rows], pa, interleaved)
    err = np.abs(_np(y)[rows] - ref)
    assert (err <= oa.rope_tolerance(ref, mag, dtype)).all(), err.max()
    z = w4.rope(x, torch.from_numpy(pos).to(cuda_device), table, pair_axes=pa, interleaved=interleaved, out=x)
    assert z is x and torch.equal(x, y)


def test_rope_table(w4, cuda_device):
    t = _np(w4.rope_table(1 << 20, 64, base=1e6, device=cuda_device))
    p, i = (1 << 20) - 1, 3
    assert abs(t[p, i] - np.cos(p * 1e6 ** (-2 * i / 64))) < 1e-7
    assert abs(t[p, 32 + i] - np.sin(p * 1e6 ** (-2 * i / 64))) < 1e-7


def test_rope_position_outside_the_table(w4, cuda_device):
    import torch

    table = w4.rope_table(10, 64, device=cuda_device)
    x = torch.randn(3, 2, 64, device=cuda_device).half()
    y = w4.rope(x, torch.tensor([1, 10, -1], dtype=torch.int32, device=cuda_device), table)
    assert w4.device_status(raise_on_error=False) == 9
    assert torch.equal(y[1:], x[1:]) and not torch.equal(y[0], x[0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,G,D", [(5, 1, 128), (8, 8, 64), (40, 8, 128)])
@pytest.mark.parametrize("lens", ["one token", "few", "short of room", "chunks", "empty"])
@pytest.mark.parametrize("layout,page", [("token", 16), ("head", 48), ("joint", 64)])
def test_append(w4, cuda_device, H, G, D, lens, layout, page, dtype):
    import torch

    b = Batch(cuda_device, dtype, H, G, D, page, LENS[lens], seed=D + page, layout=layout, poison=3.0)
    T = b.offsets[-1]
    kv = torch.randn(T, 2 * G + 1, D, device=cuda_device).to(_t(dtype))
    kn, vn = kv[:, :G], kv[:, G:2 * G]
    table = w4.rope_table(2000, D // 2, device=cuda_device)
    k0, v0 = _np(b.k), _np(b.v)
    q = w4.kv_append(kn, vn, b.k, b.v, b.page_table, b.q_offsets, b.kv_lens, q=b.q, table=table)
    _, place = oa.places(b.offsets, b.kv)
    pos = np.maximum(place, 0)[None]
    q_ref, q_mag = oa.rope(_np(b.q), _np(table), pos)
    k_ref, k_mag = oa.rope(_np(kn), _np(table), pos)
    q_ref[place < 0] = _np(b.q)[place < 0]   # no place: q as it is
    assert (np.abs(_np(q) - q_ref) <= oa.rope_tolerance(q_ref, q_mag, dtype)).all()
    where = (b.table, b.offsets, b.kv)
    tol = oa.append(np.zeros_like(k0), oa.rope_tolerance(k_ref, k_mag, dtype), *where)
    assert (np.abs(_np(b.k) - oa.append(k0, k_ref, *where)) <= tol).all()   # other slots: untouched
    assert np.array_equal(_np(b.v), oa.append(v0, _np(vn), *where))
    # without rotation, without queries: the rows themselves
    assert w4.kv_append(vn, kn, b.k, b.v, b.page_table, b.q_offsets, b.kv_lens) is None
    assert np.array_equal(_np(b.v), oa.append(v0, _np(kn), *where))


def test_append_positions_and_q_in_place(w4, cuda_device):
    import torch

    b = Batch(cuda_device, "fp16", 4, 2, 64, 16, LENS["few"], seed=23, poison=1.0)
    T = b.offsets[-1]
    r = np.random.default_rng(23)
    pos = _positions(r, 3, T, 900)
    table = w4.rope_table(900, 64, device=cuda_device)
    pa = [i % 3 for i in range(32)]
    kn = torch.randn(T, 2, 64, device=cuda_device).half()
    q = b.q.contiguous()
    q0 = _np(q)
    got = w4.kv_append(kn, kn, b.k, b.v, b.page_table, b.q_offsets, b.kv_lens, q=q, q_out=q, table=table,
                       positions=torch.from_numpy(pos).to(cuda_device), pair_axes=pa, interleaved=True)
    ref, mag = oa.rope(q0, _np(table), pos, pa, True)
    assert got is q and (np.abs(_np(q) - ref) <= oa.rope_tolerance(ref, mag, "fp16")).all()


# ---------------------------------------------------------------- refusals --

def test_nothing_to_do(w4, cuda_device):
    import torch

    b = Batch(cuda_device, "fp16", 10, 2, 128, 16, [(0, 30)], seed=24)
    assert w4.paged_attention(*b.args(), 1).shape == (0, 10, 128)
    assert w4.kv_append(b.q[:, :2], b.q[:, :2], *b.args()[1:]) is None
    assert w4.rope(b.q, torch.zeros(0, dtype=torch.int32, device=cuda_device),
                   w4.rope_table(4, 128, device=cuda_device)).shape == (0, 10, 128)


@pytest.mark.parametrize("q_len", [1, 60])
def test_bad_page_is_reported(w4, cuda_device, q_len):
    for bad in (-1, 1 << 30):
        b = Batch(cuda_device, "fp16", 10, 2, 128, 16, [(q_len, 100), (1, 50)], seed=25)
        good = w4.paged_attention(*b.args(), b.max_q)
        b.page_table[0, 2] = bad
        out = w4.paged_attention(*b.args(), b.max_q)
        assert w4.device_status(raise_on_error=False) == 9
        assert (out[q_len:] == good[q_len:]).all()   # the other sequence is served
        b.page_table[0, 6] = bad                      # the page of place 99, where a token goes
        w4.kv_append(b.q[:, :2], b.q[:, :2], *b.args()[1:])
        assert w4.device_status(raise_on_error=False) == 9


@pytest.mark.parametrize("q_len", [1, 60])
def test_bad_lengths_and_offsets_are_reported(w4, cuda_device, q_len):
    import torch

    b = Batch(cuda_device, "fp16", 10, 2, 128, 16, [(q_len, 100), (1, 50)], seed=26)
    for lens in ([100, -3], [100, 1 << 29]):
        bad = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
        b.page_table[:] = b.page_table.clamp(min=0)
        w4.paged_attention(*b.args()[:-1], bad, b.max_q)
        assert w4.device_status(raise_on_error=False) == 9
        w4.kv_append(b.q[:, :2], b.q[:, :2], *b.args()[1:-1], bad)
        assert w4.device_status(raise_on_error=False) == 9
    T = q_len + 1
    for off in ([0, T + 5, T], [1, 1, T], [0, q_len, q_len], [0, -4, T], [0, 0, T - 1], [0, q_len, T + 9]):
        bad = torch.tensor(off, dtype=torch.int32, device=cuda_device)
        w4.paged_attention(*b.args()[:-2], bad, b.kv_lens, b.max_q)
        assert w4.device_status(raise_on_error=False) in (6, 9)
        w4.kv_append(b.q[:, :2], b.q[:, :2], *b.args()[1:-2], bad, b.kv_lens)
        assert w4.device_status(raise_on_error=False) in (6, 9)


def test_too_small_max_q_len_is_reported(w4, cuda_device):
    b = Batch(cuda_device, "fp16", 10, 2, 128, 16, [(50, 100), (1, 40)], seed=27)
    good = w4.paged_attention(*b.args(), 50)
    out = w4.paged_attention(*b.args(), 1)
    assert w4.device_status(raise_on_error=False) == 6
    assert (out[50:] == good[50:]).all() or np.allclose(_np(out[50:]), _np(good[50:]), atol=2e-3)


def test_wrapper_refusals(w4, cuda_device):
    import torch

    b = Batch(cuda_device, "fp16", 10, 2, 128, 16, [(2, 30)], seed=28)
    q, k, v, pt, qo, kl = b.args()
    at = w4.paged_attention
    with pytest.raises(ValueError):
        at(q.float(), k, v, pt, qo, kl, 2)
    with pytest.raises(ValueError):
        at(q.bfloat16(), k, v, pt, qo, kl, 2)
    with pytest.raises(ValueError):
        at(q[:, :9], k, v, pt, qo, kl, 2)            # 9 heads over 2
    with pytest.raises(ValueError):
        at(q, k, v[:-1], pt, qo, kl, 2)
    with pytest.raises(ValueError):
        at(q, k, v, pt.long(), qo, kl, 2)
    with pytest.raises(ValueError):
        at(q, k, v, pt, qo[:-1], kl, 2)
    with pytest.raises(ValueError):
        at(q, k, v, pt.cpu(), qo, kl, 2)
    with pytest.raises(ValueError):
        at(q, k, v, pt, qo, kl, 2, out=torch.empty_like(q[:1]))
    for kw, status in (({"window": -1}, 1), ({"window": 8, "causal": False}, 1), ({"scale": float("nan")}, 1),
                       ({"scale": 0.0}, 1)):
        with pytest.raises(w4.W4A16Error) as e:
            at(q, k, v, pt, qo, kl, 2, **kw)
        assert e.value.status == status
    with pytest.raises(w4.W4A16Error) as e:
        at(q, k[:, :15], v[:, :15], pt, qo, kl, 2)   # a page of 15
    assert e.value.status == 2
    with pytest.raises(ValueError):
        w4.kv_append(q[:, :2], q[:, :1], k, v, pt, qo, kl)
    with pytest.raises(ValueError):
        w4.kv_append(q[:, :2], q[:, :2], k, v, pt, qo, kl, positions=torch.zeros(2, dtype=torch.int32))
    table = w4.rope_table(64, 128, device=cuda_device)
    pos = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    with pytest.raises(ValueError):
        w4.rope(q, pos[:1], table)
    with pytest.raises(ValueError):
        w4.rope(q, pos, table, pair_axes=[0] * 63)
    with pytest.raises(w4.W4A16Error):
        w4.rope(q, pos, table, pair_axes=[1] * 64)   # axis 1 of one
    with pytest.raises(w4.W4A16Error):
        w4.rope(q[..., :64], pos, table)             # a wider table than the head


def test_workspace_refusals(w4, cuda_device):
    b = Batch(cuda_device, "fp16", 10, 2, 128, 16, [(1, 3000)], seed=29)
    need = int(w4.lib().w4a16_paged_attention_workspace_bytes(1, 1, 10, 2, 128, 1))
    if need == 0:
        pytest.skip("this build needs no workspace")
    c = w4._cache(b.k, b.v, b.page_table, b.q_offsets, b.kv_lens, b.q)
    out = b.q.contiguous()

    def call(ws, n):
        return w4.lib().w4a16_paged_attention(ctypes.byref(c), 1, w4._ptr(b.q), b.q.stride(0), b.q.stride(1), 10, 1, 1,
                                              0, 0.1, w4._ptr(out), None, ws, n, None)

    assert call(None, 0) == 7
    assert call(w4._ptr(out), need - 1) == 7


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("H,G,D,page", [(10, 1, 128, 16), (10, 1, 64, 48), (24, 2, 128, 128), (32, 1, 128, 32)])
def test_some_rows_over_long_sequences(w4, cuda_device, H, G, D, page, window):
    """A few to 128 rows per cached head over thousands of places: blocks are shared out between
    the halves of a tile and between thread blocks; several tiles to a thread block."""
    r = np.random.default_rng(D + page + window)
    most = 128 // (H // G)
    lens = [(int(n), int(n + c)) for n, c in zip(r.integers(1, most + 1, 20), r.integers(0, 5000, 20))]
    b = Batch(cuda_device, "fp16", H, G, D, page, lens, seed=page)
    out, lse = w4.paged_attention(*b.args(), b.max_q, window=window, return_lse=True)
    b.check(out, lse, window=window)


@pytest.mark.parametrize("H,G,D", [(10, 1, 64), (16, 2, 128), (32, 1, 128)])
def test_some_rows_of_many_short_sequences(w4, cuda_device, H, G, D):
    """One to four blocks each: tiles of one block and of several follow each other in every order."""
    r = np.random.default_rng(H + D)
    most = 128 // (H // G)
    lens = [(int(n), int(n + c)) for n, c in zip(r.integers(0, most + 1, 260), r.integers(0, 450, 260))]
    b = Batch(cuda_device, "bf16", H, G, D, 16, lens, seed=D)
    b.check(w4.paged_attention(*b.args(), b.max_q))


def test_chunks_with_a_few_rows_in_the_last_tile(w4, cuda_device):
    """256-row tiles whose last one has 1 to 255 rows, with and without a part in another thread block."""
    lens = [(n, n + c) for n, c in ((52, 0), (53, 300), (77, 1100), (103, 40), (26, 900), (103, 3000))]
    b = Batch(cuda_device, "fp16", 10, 2, 128, 16, lens, seed=31)
    out, lse = w4.paged_attention(*b.args(), b.max_q, return_lse=True)
    b.check(out, lse)
