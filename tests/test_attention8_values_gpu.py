"""Attention over an 8-bit cache whose rows are not all ordinary numbers, on the GPU, against the 64-bit oracle
(oracle/attention.py derives the bounds): rows with an infinity or a NaN, rows of zeros, and values as large as
32 bits hold."""
import numpy as np
import pytest

from oracle import attention as oa
from test_attention8_gpu import STEP_ROWS, Batch8
from test_kv_cache8_gpu import FORMS, _normals, _numbers
from test_paged_attention_gpu import DTYPES, _np, _status_stays_clean, _t, w4  # noqa: F401

pytestmark = pytest.mark.gpu


def _agrees(b, out, lse, where, **kw):
    """out and lse of the rows and heads of `where` [T, H] are the oracle's."""
    tiles = b.max_q * b.H // b.G > STEP_ROWS
    with np.errstate(invalid="ignore"):
        ref, lse_ref, parts = oa.attention8(_np(b.q), _numbers(b.k8), _numbers(b.v8), _np(b.k_scale), _np(b.v_scale),
                                            b.table, b.offsets, b.kv, **kw)
        tol = oa.attention8_tolerance(ref, parts, b.dtype, tiles)
        lse_tol = oa.lse8_tolerance(lse_ref, b.D, parts, b.dtype)
        assert (np.abs(_np(out) - ref) <= tol)[where].all()
        assert (np.abs(_np(lse) - lse_ref) <= lse_tol)[where].all()


def _append_one(w4, b, place, k, v):  # noqa: F811
    """Rows k and v [1, G, D] at a place of the first sequence."""
    import torch

    i32 = dict(dtype=torch.int32, device=k.device)
    w4.kv_append(k, v, b.k8, b.v8, b.page_table[:1], torch.tensor([0, 1], **i32), torch.tensor([place + 1], **i32),
                 k_scale=b.k_scale, v_scale=b.v_scale)


def _with_a_bad_row(w4, dev, H, G, D, form, dtype, bad, q_len, length, window, back):  # noqa: F811
    """(batch, result with ordinary rows, result where head 0's row at place length - back has no number, which
    rows and heads see it)"""
    b = Batch8(dev, dtype, form, H, G, D, 16, [(q_len, length), (1, 50)], seed=H + D + q_len)
    place = length - back
    k, v = (_normals((1, G, D), s, _t(dtype), dev) for s in (31, 32))
    _append_one(w4, b, place, k, v)
    good = b.attend(w4, window=window, return_lse=True)
    (k if "key" in bad else v)[0, 0, 7] = float("nan") if "NaN" in bad else -float("inf")
    _append_one(w4, b, place, k, v)
    _, at = oa.places(b.offsets, b.kv)
    sees = np.zeros((q_len + 1, H), bool)
    row_sees = (at >= place) & ((at - window < place) if window else True)
    sees[:q_len, :H // G] = row_sees[:q_len, None]
    assert sees.any() and not sees.all()
    return b, good, b.attend(w4, window=window, return_lse=True), sees


BAD = ["NaN value", "infinite value", "NaN key"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len,window,back", [(3, 0, 1), (9, 0, 1), (9, 0, 5), (9, 20, 25)])
def test_few_rows_that_do_not_see_a_bad_row_keep_their_bits(w4, cuda_device, q_len, window, back, D, bad, form,  # noqa: F811
                                                            dtype):
    """The row of a later token, or one before some rows' window."""
    import torch

    _, good, got, sees = _with_a_bad_row(w4, cuda_device, 10, 2, D, form, dtype, bad, q_len, 200, window, back)
    sees = torch.from_numpy(sees).to(cuda_device)
    assert bool(got[0][sees].isnan().all())
    for x, y in zip(got, good):
        assert torch.equal(x[~sees], y[~sees])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form,D", [("int8", 128), ("e4m3", 64), ("e4m3", 128)])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("q_len,window,back", [(20, 0, 1), (20, 30, 40), (130, 0, 1), (130, 0, 70), (130, 64, 150)])
def test_tiles_keep_a_bad_row_to_the_rows_that_see_it(w4, cuda_device, q_len, window, back, bad, form, D,  # noqa: F811
                                                      dtype):
    """Rows of the same tile, and of others that work on the same block of places, do not meet it."""
    b, _, got, sees = _with_a_bad_row(w4, cuda_device, 10, 2, D, form, dtype, bad, q_len, 300, window, back)
    assert all(np.isnan(_np(x))[sees].all() for x in got)
    _agrees(b, *got, ~sees, window=window)


LEAST = {"appended": oa.LEAST / 127, "never appended": 0.0}


def _zeros_and_large(dev, lens, D, form, least, e, drop, first):
    """Zero rows and rows of scale 2^e, half of each sequence's places each, the zero rows' scores lower by `drop`."""
    import torch

    b = Batch8(dev, "bf16", form, 10, 2, D, 16, lens, seed=41)
    b.q.copy_(torch.ones_like(b.q))
    b.k8.copy_(torch.ones(b.k8.shape, device=dev).to(b.k8.dtype))
    b.k_scale.fill_(drop / D ** 0.5)
    b.v_scale.fill_(2.0 ** e)
    at = [(b.table[s][p // 16], p % 16) for s, m in enumerate(b.kv) for p in range(m) if (p < m // 2) == first]
    pages, slots = torch.tensor(at, device=dev).unbind(1)
    b.v8.view(torch.uint8)[pages, slots] = 0
    b.v_scale[pages, :, slots] = LEAST[least]
    b.k_scale[pages, :, slots] = 0
    return b


@pytest.mark.parametrize("lens", [[(1, 700)], [(3, 300), (9, 640)], [(1, 300)] * 90])
@pytest.mark.parametrize("form,least", [("int8", "appended"), ("e4m3", "never appended")])
@pytest.mark.parametrize("e,drop", [(10, 8.0), (20, 0.0), (45, 8.0), (90, 0.0)])
@pytest.mark.parametrize("first", [True, False])
def test_rows_of_zeros_count_in_the_sum(w4, cuda_device, first, e, drop, least, form, lens):  # noqa: F811
    b = _zeros_and_large(cuda_device, lens, 64, form, least, e, drop, first)
    b.check(*b.attend(w4, return_lse=True))


def _of_scale(dev, q_len, D, form, e, spread=0.0):
    """Values of scales between 2^(e - spread) and 2^e."""
    import torch

    b = Batch8(dev, "bf16", form, 10, 2, D, 16, [(q_len, 600), (1, 40)], seed=42)
    down = spread * torch.rand(b.v_scale.shape, generator=torch.Generator().manual_seed(43))
    b.v_scale.copy_(2.0 ** (e - down))
    return b


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len", [1, 9])
@pytest.mark.parametrize("e", [61, 64, 90, 103, 114, 118])
def test_few_rows_over_large_values(w4, cuda_device, e, q_len, D, form):  # noqa: F811
    """Up to the largest that 32 bits hold: the scores differ by little there, as weights below 2^-(126 - e) are lost."""
    e = min(e, 116) if form == "e4m3" else e
    b = _of_scale(cuda_device, q_len, D, form, e)
    if e > 110:
        b.q.mul_(2.0 ** -6)
    b.check(*b.attend(w4, return_lse=True))


@pytest.mark.parametrize("form,D", [("int8", 128), ("e4m3", 64), ("e4m3", 128)])
@pytest.mark.parametrize("q_len", [20, 40, 130])
@pytest.mark.parametrize("e,spread", [(62, 0), (64, 10), (70, 0), (90, 30), (116, 0)])
def test_tiles_over_large_values(w4, cuda_device, e, spread, q_len, form, D):  # noqa: F811
    b = _of_scale(cuda_device, q_len, D, form, e, spread)
    b.check(*b.attend(w4, return_lse=True))


@pytest.mark.parametrize("lens", [[(20, 700)], [(40, 700), (1, 90)], [(130, 800)]])
@pytest.mark.parametrize("form,least,D", [("int8", "appended", 128), ("e4m3", "never appended", 64)])
@pytest.mark.parametrize("e,drop", [(45, 8.0), (60, 8.0), (90, 8.0), (110, 0.0)])
@pytest.mark.parametrize("first", [True, False])
def test_rows_of_zeros_count_in_the_sum_of_tiles(w4, cuda_device, first, e, drop, least, form, D, lens):  # noqa: F811
    b = _zeros_and_large(cuda_device, lens, D, form, least, e, drop, first)
    b.check(*b.attend(w4, return_lse=True))


@pytest.mark.parametrize("form,D", [("int8", 64), ("int8", 128), ("e4m3", 128)])
@pytest.mark.parametrize("q_len", [20, 60])
def test_tiles_round_the_weights_and_the_result_alone(w4, cuda_device, q_len, D, form):  # noqa: F811
    """Errors of fp16's rounding are alike and independent, of the weights (each of a random value: as large a part of
    the result's size as of theirs) and of the result: together sqrt(2) times the latter. A third rounding would make
    it sqrt(3); the limit is between them."""
    b = Batch8(cuda_device, "fp16", form, 10, 2, D, 16, [(q_len, 1500)], seed=51)
    out, lse = b.attend(w4, return_lse=True)
    b.check(out, lse, tiles=False)
    ref, _, _ = oa.attention8(_np(b.q), _numbers(b.k8), _numbers(b.v8), _np(b.k_scale), _np(b.v_scale), b.table,
                              b.offsets, b.kv)
    alone = np.sqrt(((ref.astype(np.float16) - ref) ** 2).mean())
    assert np.sqrt(((_np(out) - ref) ** 2).mean()) <= 1.56 * alone
