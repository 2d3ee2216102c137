"""Head norms with the rotation, the append into an 8-bit cache and reading it
back, on the GPU, against the 64-bit oracle (oracle/attention.py derives the bounds)."""
import numpy as np
import pytest

from oracle import attention as oa
from test_paged_attention_gpu import DTYPES, _np, _status_stays_clean, _t, w4  # noqa: F401

pytestmark = pytest.mark.gpu

FORMS = ["int8", "e4m3"]


def _held(form):
    import torch

    return {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}[form]


def _numbers(t):
    """The values of an 8-bit (or any) tensor in 64 bits."""
    return t.float().double().cpu().numpy()


def _scaled(w4, cache, scale):
    return _numbers(cache) * np.swapaxes(_np(scale), 1, 2)[..., None]


def _normals(shape, seed, dtype=None, dev=None):
    import torch

    x = torch.randn(*shape, generator=torch.Generator().manual_seed(seed))
    return x.to(dtype).to(dev) if dtype else x.to(dev)


# ------------------------------------------------------------------- rope --

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,D,R,interleaved,axes", [
    (1, 1, 16, 16, False, 1), (5, 3, 48, 32, True, 1), (7, 5, 64, 64, False, 3), (3, 9, 80, 48, False, 2),
    (33, 18, 128, 64, True, 4), (1, 40, 128, 128, False, 1), (2, 3, 256, 256, False, 1), (3, 2, 512, 128, True, 1),
    (700, 40, 128, 128, False, 1), (400, 33, 96, 96, True, 1), (90, 17, 272, 256, False, 1)])
def test_rope_norm(w4, cuda_device, T, H, D, R, interleaved, axes, dtype):  # noqa: F811
    import torch

    dt = _t(dtype)
    fused = _normals((T, (H + 1) * D), 1, dt, cuda_device) * 3
    x = fused[:, D:].unflatten(1, (H, D))
    weight = (1 + _normals((D,), 2)).to(cuda_device)
    table = w4.rope_table(64, R, device=cuda_device)
    positions = torch.randint(0, 64, (axes, T), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    pair_axes = [i % axes for i in range(R // 2)]
    y = w4.rope(x, positions.to(cuda_device), table, pair_axes=pair_axes, interleaved=interleaved, norm=weight, eps=0.3)
    ref, mag = oa.rope(oa.head_norm(_np(x), _np(weight), np.float32(0.3)), _np(table), positions.numpy(), pair_axes,
                       interleaved)
    assert (np.abs(_np(y) - ref) <= oa.norm_rope_tolerance(ref, mag, dtype)).all()
    # in place, on the strided rows, with nothing beside them touched
    before = fused.clone()
    out = w4.rope(x, positions.to(cuda_device), table, pair_axes=pair_axes, interleaved=interleaved, norm=weight,
                  eps=0.3, out=x)
    assert out is x and torch.equal(x, y) and torch.equal(fused[:, :D], before[:, :D])


def test_rope_norm_of_small_and_large_heads(w4, cuda_device):  # noqa: F811
    """The squares of bf16's largest numbers pass 32 bits: such heads come out as 0 or NaN, as in 32 bits; those up to
    2^60 do not. Heads of zeros stay zero."""
    import torch

    x = torch.ones(4, 1, 64, dtype=torch.bfloat16, device=cuda_device)
    for i, e in enumerate((-60, 0, 30, 60)):
        x[i] *= 2.0 ** e
    x[1] = 0
    weight, table = torch.full((64,), 0.5, device=cuda_device), w4.rope_table(4, 64, device=cuda_device)
    y = w4.rope(x, torch.zeros(4, dtype=torch.int32, device=cuda_device), table, norm=weight, eps=1e-30)
    want = [2.0 ** -60 / np.sqrt(2.0 ** -120 + 1e-30) / 2, 0.0, 0.5, 0.5]
    assert np.allclose(_np(y)[:, 0, 0], want, rtol=2.0 ** -8)
    assert w4.rope(x[:0], torch.zeros(0, dtype=torch.int32, device=cuda_device), table, norm=weight).shape == (0, 1, 64)


def test_rope_norm_reports_positions(w4, cuda_device):  # noqa: F811
    """A position outside the table: the head is normalised and not turned."""
    import torch

    x = _normals((3, 2, 64), 5, torch.float16, cuda_device)
    weight, table = torch.ones(64, device=cuda_device), w4.rope_table(4, 64, device=cuda_device)
    y = w4.rope(x, torch.tensor([0, 4, -1], dtype=torch.int32, device=cuda_device), table, norm=weight)
    assert w4.device_status(raise_on_error=False) == 9
    ref = oa.head_norm(_np(x), np.ones(64), 1e-6)
    assert (np.abs(_np(y) - ref) <= oa.norm_rope_tolerance(ref, np.abs(ref), "fp16")).all()


# ----------------------------------------------------------------- append --

class Rows:
    """A call's rows, and a cache of zeros with room for them: lens is a list of (new tokens, cached ones with them)."""

    def __init__(self, w4, dev, dtype, form, H, G, D, page, lens, seed=0, layout="token", gain=1.0):  # noqa: F811
        import torch

        self.w4, self.form, self.dtype = w4, form, dtype
        q_lens, self.kv = [n for n, _ in lens], [m for _, m in lens]
        self.offsets = np.concatenate([[0], np.cumsum(q_lens)]).astype(int).tolist()
        T = self.offsets[-1]
        need = [-(-m // page) for m in self.kv]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        self.table = [[-1] * (max(need + [1]) + 1) for _ in lens]
        at = 0
        for b, n in enumerate(need):
            self.table[b][:n] = order[at:at + n]
            at += n
        held = _held(form) if form else _t(dtype)
        if layout == "head":  # heads of a page after one another; scales among others
            caches = [torch.zeros(pages, G, page, D, dtype=torch.uint8 if form else held, device=dev) for _ in range(2)]
            caches = [(c.view(held) if form else c).transpose(1, 2) for c in caches]
            joint = torch.zeros(pages, 2, G, page, device=dev)
            self.ks, self.vs = joint[:, 0], joint[:, 1]
        else:
            caches = [torch.zeros(pages, page, G, D, dtype=torch.uint8 if form else held, device=dev) for _ in range(2)]
            caches = [c.view(held) if form else c for c in caches]
            self.ks, self.vs = (torch.zeros(pages, G, page, device=dev) for _ in range(2))
        self.k_cache, self.v_cache = caches
        if not form:
            self.ks = self.vs = None
        self.fused = _normals((T, (H + 2 * G) * D), seed + 1, _t(dtype), dev) * gain
        self.q, self.k, self.v = (x.unflatten(1, (-1, D)) for x in self.fused.split([H * D, G * D, G * D], 1))
        self.args = [torch.tensor(x, dtype=torch.int32, device=dev) for x in (self.table, self.offsets, self.kv)]
        self.T, self.page = T, page

    def append(self, **kw):
        return self.w4.kv_append(self.k, self.v, self.k_cache, self.v_cache, *self.args, k_scale=self.ks,
                                 v_scale=self.vs, **kw)

    def read(self, rows=None, **kw):
        return self.w4.kv_read(self.k_cache, self.v_cache, *self.args, self.T if rows is None else rows,
                               k_scale=self.ks, v_scale=self.vs, **kw)

    def stored(self, cache, scale):
        """What the cache holds at the rows' places, and the scales; NaN where a row has no place."""
        values, scales = _numbers(cache), None if scale is None else _np(scale)
        G, D = values.shape[2:]
        out, of = np.full((self.T, G, D), np.nan), np.full((self.T, G), np.nan)
        for t, (b, p) in enumerate(zip(*oa.places(self.offsets, self.kv))):
            if p >= 0:
                at = self.table[b][p // self.page], p % self.page
                out[t] = values[at]
                if scale is not None:
                    of[t] = scales[at[0], :, at[1]]
                    out[t] *= of[t][:, None]
        return out, of


LENS = {
    "steps": [(1, 1), (1, 16), (1, 17), (1, 300), (1, 49)],
    "chunks": [(40, 40), (0, 9), (1, 5), (23, 130), (7, 49)],
    "short of room": [(7, 4), (3, 0), (2, 40), (0, 0)],
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", [None, *FORMS])
@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("H,G,D,page,layout", [(5, 1, 128, 16, "token"), (8, 8, 64, 48, "head"),
                                               (9, 3, 64, 16, "token"), (40, 8, 128, 32, "head")])
def test_append(w4, cuda_device, H, G, D, page, layout, lens, form, dtype):  # noqa: F811
    r = Rows(w4, cuda_device, dtype, form, H, G, D, page, LENS[lens], seed=D + H, layout=layout)
    qw, kw = ((1 + _normals((D,), s)).to(cuda_device) for s in (7, 8))
    table = w4.rope_table(512, D // 2, device=cuda_device)
    q = r.append(q=r.q, table=table, q_norm=qw, k_norm=kw, eps=1e-5)
    seq, place = oa.places(r.offsets, r.kv)
    ok = place >= 0

    def turned(x, weight):
        x = oa.head_norm(_np(x), _np(weight), np.float32(1e-5))
        y, mag = oa.rope(x, _np(table), np.maximum(place, 0)[None])
        y[~ok], mag[~ok] = x[~ok], np.abs(x[~ok])
        return y, mag

    ref, mag = turned(r.q, qw)
    assert (np.abs(_np(q) - ref) <= oa.norm_rope_tolerance(ref, mag, dtype)).all()
    for x, cache, scale, (ref, mag) in ((r.k, r.k_cache, r.ks, turned(r.k, kw)),
                                        (r.v, r.v_cache, r.vs, (_np(r.v), None))):
        got, scales = r.stored(cache, scale)
        off = 0.0 if mag is None else oa.NORM * np.abs(ref) + (2.0 ** -22 + oa.NORM) * mag
        if form:
            tol, s_tol = oa.held_tolerance(ref, form, off)
            s_ref = np.maximum(np.abs(ref).max(-1), oa.LEAST) / oa.MOST[form]
            assert (np.abs(scales - s_ref)[ok] <= s_tol[ok]).all()
        else:
            tol = 0.0 if mag is None else oa.norm_rope_tolerance(ref, mag, dtype)
        assert (np.abs(got - ref) <= tol)[ok].all()
        # nothing else is written
        assert (_numbers(cache) != 0).any(-1).sum() <= ok.sum() * G
        if form:
            assert (_np(scale) != 0).sum() == ok.sum() * G


@pytest.mark.parametrize("form", FORMS)
def test_append_without_norm_or_rotation(w4, cuda_device, form):  # noqa: F811
    """Keys and values as they are: the scales are exact, and the rows the nearest that the format has."""
    r = Rows(w4, cuda_device, "bf16", form, 4, 4, 128, 16, [(200, 200), (130, 177)], seed=4)
    assert r.append() is None
    for x, cache, scale in ((r.k, r.k_cache, r.ks), (r.v, r.v_cache, r.vs)):
        got, scales = r.stored(cache, scale)
        top = np.abs(_np(x)).max(-1)
        assert np.array_equal(scales.astype(np.float32), top.astype(np.float32) / np.float32(oa.MOST[form]))
        tol, _ = oa.held_tolerance(_np(x), form)
        assert (np.abs(got - _np(x)) <= tol).all()
        assert np.array_equal(np.abs(got / scales[..., None]).max(-1).round(3), np.full(top.shape, oa.MOST[form]))


@pytest.mark.parametrize("form", FORMS)
def test_rows_of_zeros_small_large_and_no_numbers(w4, cuda_device, form):  # noqa: F811
    r = Rows(w4, cuda_device, "bf16", form, 1, 1, 64, 16, [(8, 8)])
    r.k[:] = 0
    r.k[1] = 2.0 ** -120
    r.k[2, 0, 5] = 3.0e38
    r.k[3, 0, 7] = float("inf")
    r.k[4, 0, 9] = float("nan")
    r.k[5, 0, 63] = -float("inf")
    r.k[6, 0, 0] = -(2.0 ** -100)
    r.append()
    got, scales = r.stored(r.k_cache, r.ks)
    assert not got[0].any() and scales[0] > 0 and not got[1].any() and not got[7].any()
    assert np.isclose(got[2, 0, 5], _np(r.k)[2, 0, 5], rtol=2.0 ** -20) and not np.delete(got[2, 0], 5).any()
    assert np.isnan(got[3:6]).all() and np.isnan(scales[3:6]).all()
    assert np.isclose(got[6, 0, 0], -(2.0 ** -100), rtol=2.0 ** -20)
    for dtype in DTYPES:
        k, _ = r.read(dtype=_t(dtype))
        k = _np(k)
        assert np.isnan(k[3:6]).all() and not k[[0, 1, 7]].any()
        assert k[2, 0, 5] == (np.inf if dtype == "fp16" else float(_t_round(got[2, 0, 5])))


def _t_round(x):
    import torch

    return torch.tensor(x, dtype=torch.float32).to(torch.bfloat16).double()


# ------------------------------------------------------------------- read --

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", [None, *FORMS])
@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("G,D,page,layout", [(1, 128, 16, "token"), (3, 64, 48, "head"), (8, 128, 16, "head")])
def test_read(w4, cuda_device, G, D, page, layout, lens, form, dtype):  # noqa: F811
    import torch

    r = Rows(w4, cuda_device, dtype, form, 1, G, D, page, LENS[lens], seed=G, layout=layout)
    r.append()
    seq, place = oa.places(r.offsets, r.kv)
    ok = place >= 0
    k, v = r.read(dtype=_t(dtype))
    for x, got, cache, scale in ((r.k, k, r.k_cache, r.ks), (r.v, v, r.v_cache, r.vs)):
        assert got.dtype == _t(dtype) and got.is_contiguous()
        held, _ = r.stored(cache, scale)
        assert not _np(got)[~ok].any()
        if form:
            # one fp32 product, rounded to the type
            tol = (oa.UNIT[dtype] + 2.0 ** -23) * np.abs(held) + oa.TINY[dtype]
            assert (np.abs(_np(got) - held) <= tol)[ok].all()
        else:
            assert torch.equal(got[torch.from_numpy(ok).to(got.device)], x[torch.from_numpy(ok).to(got.device)])
    into = [torch.empty_like(k), torch.empty_like(v)]
    again = r.read(k_out=into[0], v_out=into[1])
    assert again[0] is into[0] and torch.equal(into[0], k) and torch.equal(into[1], v)


def test_read_a_prefix(w4, cuda_device):  # noqa: F811
    """Places [0, 37) of one sequence and [5, 21) of another, through another batch's offsets and lengths."""
    import torch

    r = Rows(w4, cuda_device, "fp16", "int8", 1, 2, 64, 16, [(50, 50), (33, 33)], seed=9)
    r.append()
    all_k, all_v = r.read(dtype=torch.float16)
    i32 = dict(dtype=torch.int32, device=cuda_device)
    k, v = w4.kv_read(r.k_cache, r.v_cache, r.args[0], torch.tensor([0, 37, 53], **i32), torch.tensor([37, 21], **i32),
                      53, dtype=torch.float16, k_scale=r.ks, v_scale=r.vs)
    at = torch.tensor([*range(37), *range(55, 71)], device=cuda_device)
    assert torch.equal(k, all_k[at]) and torch.equal(v, all_v[at])


@pytest.mark.parametrize("form", FORMS)
def test_bad_pages_lengths_and_rows(w4, cuda_device, form):  # noqa: F811
    """A page entry outside the cache, a length that the table cannot name, rows behind the last sequence: reported,
    nothing stored, zeros read (rows that no sequence holds are left as they were)."""
    import torch

    for what, status in (("page", 9), ("length", 9), ("rows", 6)):
        r = Rows(w4, cuda_device, "fp16", form, 2, 1, 64, 16, [(3, 20), (2, 2)], seed=11)
        if what == "page":
            r.args[0][0, 1] = 99
        elif what == "length":
            r.args[2][0] = 1000
        else:
            r.args[1][2] = 4  # one row fewer than the call's
        r.append(q=r.q, q_norm=torch.ones(64, device=cuda_device))
        assert w4.device_status(raise_on_error=False) == status
        written = (_np(r.ks) != 0).sum()
        assert written == {"page": 2, "length": 2, "rows": 4}[what]
        k = torch.full((5, 1, 64), 7.0, dtype=torch.float16, device=cuda_device)
        r.read(k_out=k, v_out=k.clone())
        assert w4.device_status(raise_on_error=False) == status
        rows = _np(k)[:, 0]
        if what == "rows":
            assert (rows[4] == 7).all() and (rows[:4] != 7).any(-1).all()
        else:
            assert not rows[:3].any() and rows[3:].any(-1).all()


def test_prompt_then_tokens(w4, cuda_device):  # noqa: F811
    """A long call (four heads to a thread) and the same rows one at a time leave the same cache and queries."""
    import torch

    n = 1500
    whole = Rows(w4, cuda_device, "fp16", "int8", 8, 2, 128, 16, [(n, n)], seed=3)
    one = Rows(w4, cuda_device, "fp16", "int8", 8, 2, 128, 16, [(n, n)], seed=3)
    norm = (1 + 0.1 * _normals((128,), 5)).to(cuda_device)
    table = w4.rope_table(n, 128, device=cuda_device)
    how = dict(table=table, q_norm=norm, k_norm=norm)
    q = whole.append(q=whole.q, **how)
    i32 = dict(dtype=torch.int32, device=cuda_device)
    offsets = torch.tensor([0, 1], **i32)
    for t in [*range(40), n - 1]:
        got = w4.kv_append(one.k[t:t + 1], one.v[t:t + 1], one.k_cache, one.v_cache, one.args[0], offsets,
                           torch.tensor([t + 1], **i32), q=one.q[t:t + 1], k_scale=one.ks, v_scale=one.vs, **how)
        assert torch.equal(got, q[t:t + 1])
    for a, b in ((one.k_cache, whole.k_cache), (one.v_cache, whole.v_cache), (one.ks, whole.ks), (one.vs, whole.vs)):
        a, b = (x.transpose(1, 2) if x.ndim == 3 else x for x in (a, b))
        for t in [*range(40), n - 1]:
            at = one.table[0][t // 16], t % 16
            assert torch.equal(a[at], b[at])
