"""The oracle of the head norms and the 8-bit cache, pinned by closed forms."""
import numpy as np
import pytest

from oracle import attention as oa


def test_head_norm_by_hand():
    y = oa.head_norm([[3.0, -4.0]], [2.0, 1.0], 0.0)
    assert np.allclose(y, [[6.0 / np.sqrt(12.5), -4.0 / np.sqrt(12.5)]], rtol=1e-15)
    assert np.allclose(oa.head_norm([[0.0, 0.0]], [1.0, 1.0], 1e-6), 0.0)
    # eps takes half of the mean square away from the divisor's reach: 1 / sqrt(1 + 3) = 1/2
    assert np.allclose(oa.head_norm([[1.0, -1.0]], [1.0, 1.0], 3.0), [[0.5, -0.5]], rtol=1e-15)


def test_every_e4m3_number_is_its_own():
    import torch

    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    numbers = codes[np.isfinite(codes)]
    assert len(numbers) == 254 and numbers.max() == 448
    assert np.array_equal(oa.e4m3(numbers), numbers)
    middles = (np.sort(np.unique(numbers))[1:] + np.sort(np.unique(numbers))[:-1]) / 2
    away = oa.e4m3(middles * (1 + 1e-12))
    assert np.array_equal(np.abs(away), np.where(middles > 0, np.sort(np.unique(numbers))[1:],
                                                 -np.sort(np.unique(numbers))[:-1]))


@pytest.mark.parametrize("form", ["int8", "e4m3"])
def test_hold(form):
    r = np.random.default_rng(1)
    x = r.normal(size=(50, 64)) * np.exp(r.normal(size=(50, 1)))
    q, s = oa.hold(x, form)
    assert np.array_equal(np.abs(q).max(-1), np.full(50, oa.MOST[form]))
    tol, s_tol = oa.held_tolerance(x, form)
    assert (np.abs(q * s[:, None] - x) <= tol).all()
    assert (s_tol <= 2.0 ** -21 * s).all()
    # a step further is out of tolerance for integers
    if form == "int8":
        assert (np.abs((q + np.where(q >= 0, -1, 1)) * s[:, None] - x) > tol).mean() > 0.95
    q, s = oa.hold(np.zeros((1, 16)), form)
    assert not q.any() and s[0] == 2.0 ** -100 / oa.MOST[form]


def test_attention8_is_attention_of_the_rows_it_stands_for():
    r = np.random.default_rng(2)
    k, v = r.integers(-127, 128, (2, 3, 16, 1, 4))
    ks, vs = np.exp(r.normal(size=(2, 3, 1, 16))) / 127
    q = r.normal(size=(2, 2, 4))
    out, lse, parts = oa.attention8(q, k, v, ks, vs, [[2, 0]], [0, 2], [20])
    rows = [k[p, s, 0] * ks[p, 0, s] for p, s in [(2, i) for i in range(16)] + [(0, i) for i in range(4)]]
    vals = [v[p, s, 0] * vs[p, 0, s] for p, s in [(2, i) for i in range(16)] + [(0, i) for i in range(4)]]
    a = np.array([q[1, 1] @ x for x in rows]) * 0.5
    w = np.exp(a - a.max())
    assert np.allclose(out[1, 1], (w / w.sum()) @ np.array(vals), rtol=1e-12)
    assert np.isclose(lse[1, 1], a.max() + np.log(w.sum()))
    assert (parts["V"] >= 0.99 * np.abs(np.array(vals)).sum(0)).all()
