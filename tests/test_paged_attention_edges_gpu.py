"""Edges of the attention operators: lengths, windows, positions and values at which a result could
go wrong without a report."""
import numpy as np
import pytest

from oracle import attention as oa
from test_paged_attention_gpu import Batch, _np, _t

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import w4a16_group_quantized_linear_gb300 as w4

    w4.lib()
    return w4


@pytest.fixture(autouse=True)
def _status_stays_clean(w4, cuda_device):
    yield
    assert w4.device_status(raise_on_error=False) == 0


@pytest.mark.parametrize("window", [(1 << 30) + 1, (1 << 31) - 2, (1 << 31) - 1])
@pytest.mark.parametrize("lens", [[(7, 4), (2, 40), (1, 128)], [(130, 40), (57, 300), (3, 1)]])
def test_window_as_large_as_it_can_be(w4, cuda_device, lens, window):
    """No limit, also where a sequence is shorter than its new tokens."""
    b = Batch(cuda_device, "fp16", 10, 2, 128, 16, lens, seed=5)
    out, lse = w4.paged_attention(*b.args(), b.max_q, window=window, return_lse=True)
    b.check(out, lse)


@pytest.mark.parametrize("positions", [False, True])
@pytest.mark.parametrize("q_len", [1, 5, 60])
@pytest.mark.parametrize("length", [-3, 7 * 16 + 1, 7 * 16 + 60, 1 << 29])
def test_append_stores_nothing_for_a_length_out_of_range(w4, cuda_device, length, q_len, positions):
    """Its page table has room for 7 pages of 16; the other sequences' rows are stored."""
    import torch

    b = Batch(cuda_device, "fp16", 4, 2, 64, 16, [(2, 30), (q_len, 96), (3, 40)], seed=q_len, poison=3.0)
    b.page_table[1] = b.page_table[1].clamp(min=0)   # every entry names a page
    bad = torch.tensor([30, length, 40], dtype=torch.int32, device=cuda_device)
    T = b.offsets[-1]
    kn, vn = (torch.randn(T, 2, 64, device=cuda_device).half() for _ in range(2))
    want_k, want_v = b.k.clone(), b.v.clone()
    for s in (0, 2):
        for t in range(b.offsets[s], b.offsets[s + 1]):
            p = b.kv[s] - (b.offsets[s + 1] - t)
            want_k[b.table[s][p // 16], p % 16], want_v[b.table[s][p // 16], p % 16] = kn[t], vn[t]
    rotary = {}
    if positions:   # position 0 turns by nothing
        rotary = dict(table=w4.rope_table(8, 64, device=cuda_device),
                      positions=torch.zeros(T, dtype=torch.int32, device=cuda_device))
    w4.kv_append(kn, vn, b.k, b.v, b.page_table, b.q_offsets, bad, **rotary)
    assert w4.device_status(raise_on_error=False) == 9
    assert torch.equal(b.k, want_k) and torch.equal(b.v, want_v)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("window", [1, 30, 200])
@pytest.mark.parametrize("lens", [[(1, 300), (3, 200)], [(20, 400), (7, 300), (20, 100)], [(130, 500), (1, 90), (70, 1000)]])
def test_places_before_every_window_may_hold_anything(w4, cuda_device, lens, window, page):
    """Also in a page that holds places that rows see: infinities and NaN there reach no result."""
    for value in (float("nan"), float("inf")):
        b = Batch(cuda_device, "fp16", 10, 2, 128, page, lens, seed=page)
        for s, m in enumerate(b.kv):
            n = b.offsets[s + 1] - b.offsets[s]
            for p in range(max(0, m - n - window + 1)):
                b.k[b.table[s][p // page], p % page] = value
                b.v[b.table[s][p // page], p % page] = value
        out, lse = w4.paged_attention(*b.args(), b.max_q, window=window, return_lse=True)
        b.check(out, lse, window=window)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("window", [1, 30, 200])
@pytest.mark.parametrize("lens", [[(1, 300), (3, 200)], [(20, 400), (7, 300), (20, 100)], [(130, 500), (1, 90), (70, 1000)]])
def test_places_before_every_window_may_hold_anything(w4, cuda_device, lens, window, page):
    """Also in a page that holds places that rows see: infinities and NaN there reach no result."""
    for value in (float("nan"), float("inf")):
        b = Batch(cuda_device, "fp16", 10, 2, 128, page, lens, seed=page)
        for s, m in enumerate(b.kv):
            n = b.offsets[s + 1] - b.offsets[s]
            for p in range(max(0, m - n - window + 1)):
                b.k[b.table[s][p // page], p % page] = value
                b.v[b.table[s][p // page], p % page] = value
        out, lse = w4.paged_attention(*b.args(), b.max_q, window=window, return_lse=True)
        b.check(out, lse, window=window)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pattern", ["cycle", "blocks"])
@pytest.mark.parametrize("R", [32, 64])
def test_a_position_outside_the_table_leaves_only_its_own_pairs(w4, cuda_device, R, pattern, interleaved):
    """With several axes, pairs of the other axes are turned all the same; in the append too, where
    keys under the caller's positions are checked along with the queries."""
    import torch

    r = np.random.default_rng(R)
    b = Batch(cuda_device, "fp16", 4, 2, 64, 16, [(1, 20), (6, 31)], seed=R, poison=2.0)
    T, half = b.offsets[-1], R // 2
    axes = [i % 3 if pattern == "cycle" else i * 3 // half for i in range(half)]
    pos = r.integers(0, 50, (3, T)).astype(np.int32)
    pos[1, 2], pos[2, 4], pos[:, 5] = 50, -1, 1 << 30
    wrong = (pos < 0) | (pos >= 50)
    table = w4.rope_table(50, R, device=cuda_device)
    where = dict(table=table, positions=torch.from_numpy(pos).to(cuda_device), pair_axes=axes, interleaved=interleaved)

    def check(y, x):
        ref, mag = oa.rope(_np(x), _np(table), np.where(wrong, 0, pos), axes, interleaved)
        for i in range(half):
            e = [2 * i, 2 * i + 1] if interleaved else [i, i + half]
            for t in np.flatnonzero(wrong[axes[i]]):
                ref[t][:, e], mag[t][:, e] = _np(x)[t][:, e], 0
                assert np.array_equal(_np(y)[t][:, e], ref[t][:, e])
        assert (np.abs(_np(y) - ref) <= oa.rope_tolerance(ref, mag, "fp16")).all()

    check(w4.rope(b.q, where["positions"], table, pair_axes=axes, interleaved=interleaved), b.q)
    assert w4.device_status(raise_on_error=False) == 9
    kn = torch.randn(T, 2, 64, device=cuda_device).half()
    q = w4.kv_append(kn, kn, b.k, b.v, b.page_table, b.q_offsets, b.kv_lens, q=b.q, **where)
    assert w4.device_status(raise_on_error=False) == 9
    seq, place = oa.places(b.offsets, b.kv)
    pages = torch.tensor([b.table[s][p // 16] for s, p in zip(seq, place)], device=cuda_device)
    slots = torch.from_numpy(place % 16).to(cuda_device)
    check(q, b.q)
    check(b.k[pages, slots], kn)
    assert torch.equal(b.v[pages, slots], kn)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[(1, 300), (1, 5), (1, 40)], [(1, 9000), (2, 7)], [(20, 1500), (5, 20)],
                                  [(20, 6000), (5, 20)], [(130, 700), (70, 90)], [(300, 9000)]])
def test_a_query_that_is_not_a_number(w4, cuda_device, lens, D):
    """Its row's result and logarithm are NaN, and no other row changes."""
    import torch

    b = Batch(cuda_device, "fp16", 10, 2, D, 16, lens, seed=D)
    good, good_lse = w4.paged_attention(*b.args(), b.max_q, return_lse=True)
    rows = [(0, 3), (b.offsets[-1] - 1, 9)]
    other = torch.ones(b.offsets[-1], 10, dtype=torch.bool, device=cuda_device)
    for t, h in rows:
        b.q[t, h, 5] = float("nan")
        other[t, h] = False
    out, lse = w4.paged_attention(*b.args(), b.max_q, return_lse=True)
    for t, h in rows:
        assert out[t, h].isnan().all() and lse[t, h].isnan()
    assert torch.equal(out[other], good[other]) and torch.equal(lse[other], good_lse[other])


@pytest.mark.parametrize("D", [64, 128])
def test_large_bf16_values_under_rising_scores(w4, cuda_device, D):
    """Values of 10^32: the sums before their division stay finite although the running maximum lags."""
    import torch

    b = Batch(cuda_device, "bf16", 10, 2, D, 16, [(64, 256)] * 60, seed=D)   # two blocks and more for each SM
    for s, m in enumerate(b.kv):
        for p in range(0, m, 16):
            # 1/4 more in the exponent of two with each place
            b.k[b.table[s][p // 16]] = (0.25 * 0.6931 * D ** -0.5 * torch.arange(p, p + 16.0)).to(b.k)[:, None, None]
    b.q.copy_(torch.ones_like(b.q))
    b.v.mul_(1e32)
    out, lse = w4.paged_attention(*b.args(), b.max_q, return_lse=True)
    b.check(out, lse)


@pytest.mark.parametrize("lens", [[(1, 9000), (1, 300)], [(300, 4000)]])
def test_calls_after_a_wait_that_gave_up(w4, cuda_device, monkeypatch, lens):
    """Reading the timeout makes the kept workspaces ready again (test-hooks build: a 1 ms limit and a
    loader that stops after up to three blocks)."""
    import ctypes

    from w4a16_group_quantized_linear_gb300 import build

    lib = ctypes.CDLL(build.build(variant="testhooks"))
    for name, (res, args) in w4.EXPORTS.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    lib.w4a16_test_set_hooks.restype = ctypes.c_int32
    lib.w4a16_test_set_hooks.argtypes = [ctypes.c_uint64, ctypes.c_int32]
    monkeypatch.setattr(w4, "_lib", lib)
    monkeypatch.setattr(w4, "_ws", {})
    stopped = Batch(cuda_device, "fp16", 10, 2, 128, 16, [(300, 4000)], seed=1)
    b = Batch(cuda_device, "fp16", 10, 2, 128, 16, lens, seed=2)
    try:
        for limit in (0, 1, 2, 3):
            assert lib.w4a16_test_set_hooks(1_000_000, limit) == 0
            w4.paged_attention(*stopped.args(), stopped.max_q)
            assert w4.device_status(raise_on_error=False) == 5
    finally:
        assert lib.w4a16_test_set_hooks(2_000_000_000, -1) == 0
    for _ in range(2):
        b.check(w4.paged_attention(*b.args(), b.max_q))
        stopped.check(w4.paged_attention(*stopped.args(), stopped.max_q))
    assert w4.device_status(raise_on_error=False) == 0
