"""Pins of the 64-bit attention oracle: closed forms, and planted mistakes that
the pins catch."""
import numpy as np
import pytest

from oracle import attention as oa

RNG = np.random.default_rng


def _table(rows, dim, base=10000.0):
    a = np.arange(rows)[:, None] * base ** (-np.arange(0, dim, 2) / dim)
    return np.concatenate([np.cos(a), np.sin(a)], axis=1)


def _cache(r, pages=6, size=16, G=2, D=8):
    return r.normal(size=(pages, size, G, D)), r.normal(size=(pages, size, G, D))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_keeps_lengths_and_depends_on_differences(interleaved):
    r = RNG(0)
    q, k = r.normal(size=(1, 1, 32)), r.normal(size=(1, 1, 32))
    tab = _table(200, 32)

    def dot(i, j):
        a, _ = oa.rope(q, tab, [[i]], interleaved=interleaved)
        b, _ = oa.rope(k, tab, [[j]], interleaved=interleaved)
        assert np.isclose((a ** 2).sum(), (q ** 2).sum())
        return float((a * b).sum())

    assert np.isclose(dot(5, 3), dot(105, 103)) and np.isclose(dot(0, 0), float((q * k).sum()))
    assert not np.isclose(dot(5, 3), dot(3, 5))


def test_rope_by_hand():
    # a quarter turn takes (1, 0) to (0, 1) and (0, 1) to (-1, 0)
    tab = np.array([[1.0, 1.0, 0.0, 0.0], [0.0, 1.0, 1.0, 0.0]])
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    y, _ = oa.rope(x, tab, [[1]])
    assert np.array_equal(y[0, 0], [-3.0, 2.0, 1.0, 4.0, 9.0])
    y, _ = oa.rope(x, tab, [[1]], interleaved=True)
    assert np.array_equal(y[0, 0], [-2.0, 1.0, 3.0, 4.0, 9.0])
    # each pair by its own axis: axis 1 stands still
    tab = np.array([[1.0, 1.0, 0.0, 0.0], [0.0, 0.0, 1.0, 1.0]])
    y, _ = oa.rope(x, tab, [[1], [0]], pair_axes=[0, 1])
    assert np.array_equal(y[0, 0], [-3.0, 2.0, 1.0, 4.0, 9.0])


def test_places_and_append():
    seq, place = oa.places([0, 2, 2, 5], [10, 4, 1])
    assert seq.tolist() == [0, 0, 2, 2, 2] and place.tolist() == [8, 9, -2, -1, 0]
    cache = np.zeros((3, 4, 1, 1))
    got = oa.append(cache, np.arange(1, 6).reshape(5, 1, 1), [[2, 0, 1], [0, 0, 0], [1, 0, 0]], [0, 2, 2, 5],
                    [10, 4, 1])
    want = np.zeros((3, 4, 1, 1))
    want[1, 0], want[1, 1] = 1, 2   # places 8, 9 of sequence 0: page 2 of its row
    want[1, 0] = 5                  # place 0 of sequence 2 shares that page here
    assert np.array_equal(got, want)


def test_equal_keys_average_the_values():
    r = RNG(1)
    k, v = _cache(r)
    k[:] = k[0, 0, 0, 0]
    table = [[4, 2, 0]]
    q = r.normal(size=(3, 4, 8))
    out, lse, parts = oa.attention(q, k, v, table, [0, 3], [40])
    flat = oa.gather(v, table, 0, 40)
    for t in range(3):
        for h in range(4):
            assert np.allclose(out[t, h], flat[:38 + t, h // 2].mean(0))
            assert np.isclose(lse[t, h], np.log(38 + t) + 8 ** -0.5 * q[t, h].sum() * k[0, 0, 0, 0])
    assert parts["m"].tolist() == [38, 39, 40]


def test_window_and_whole_and_empty_rows():
    r = RNG(2)
    k, v = _cache(r)
    table = [[1, 3, 5], [0, 2, 4]]
    q = r.normal(size=(5, 2, 8))
    # a window of one sees the row's own place alone
    out, lse, _ = oa.attention(q, k, v, table, [0, 2, 5], [33, 2], window=1)
    assert np.allclose(out[0, 1], v[3, 15, 1]) and np.allclose(out[1, 1], v[5, 0, 1])
    # sequence 1 has two places for three new tokens: its first row sees nothing
    assert np.all(out[2] == 0) and np.all(np.isneginf(lse[2])) and np.allclose(out[3, 0], v[0, 0, 0])
    # without the causal mask every row sees the same places
    whole, _, _ = oa.attention(np.repeat(q[:1], 2, 0), k, v, table[:1], [0, 2], [33], causal=False)
    assert np.allclose(whole[0], whole[1])


def test_one_large_score_takes_all():
    k, v = np.zeros((1, 16, 1, 4)), RNG(3).normal(size=(1, 16, 1, 4))
    k[0, 7, 0, 2] = 500.0
    out, lse, _ = oa.attention(np.array([[[0, 0, 10.0, 0]]]), k, v, [[0]], [0, 1], [16])
    assert np.allclose(out[0, 0], v[0, 7, 0]) and np.isclose(lse[0, 0], 2500.0)


MUTANTS = {
    "causal mask one short": ("p + 1) if causal", "p) if causal"),
    "window one too wide": ("max(0, p - window + 1)", "max(0, p - window)"),
    "heads grouped by remainder": ("g = h // (H // G)", "g = h % G"),
    "scale dropped": ("s = scale * (k[:, g] @ q[t, h])", "s = k[:, g] @ q[t, h]"),
    "place ignores the new tokens": ("place.append(n - count + i)", "place.append(i)"),
    "sine's sign": ("x[t, :, a] * c - x[t, :, b] * s", "x[t, :, a] * c + x[t, :, b] * s"),
    "pairs always adjacent": ("(2 * i, 2 * i + 1) if interleaved else (i, i + half)", "(2 * i, 2 * i + 1)"),
    "axes ignored": ("0 if pair_axes is None else pair_axes[i]", "0"),
    "slot of the wrong page": ("page_table[b][j // size], j % size) for j", "page_table[b][0], j % size) for j"),
}


@pytest.mark.parametrize("name", sorted(MUTANTS))
def test_pins_catch_planted_mistake(name, monkeypatch):
    import types

    src = open(oa.__file__).read()
    old, new = MUTANTS[name]
    assert old in src
    bad = types.ModuleType("bad")
    exec(compile(src.replace(old, new), "bad", "exec"), bad.__dict__)
    for f in ("rope", "places", "append", "gather", "attention"):
        monkeypatch.setattr(oa, f, getattr(bad, f))
    pins = [(test_rope_keeps_lengths_and_depends_on_differences, (False,)), (test_rope_by_hand, ()),
            (test_places_and_append, ()), (test_equal_keys_average_the_values, ()),
            (test_window_and_whole_and_empty_rows, ()), (test_one_large_score_takes_all, ())]
    failed = 0
    for pin, args in pins:
        try:
            pin(*args)
        except Exception:  # noqa: BLE001 - any failure catches the mistake
            failed += 1
    assert failed
