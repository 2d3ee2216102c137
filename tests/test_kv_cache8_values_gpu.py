"""Head norms of rows whose squares 32 bits do not hold, on the GPU, against the 64-bit oracle."""
import numpy as np
import pytest

from oracle import attention as oa
from test_kv_cache8_gpu import FORMS, Rows, _normals
from test_paged_attention_gpu import _np, _status_stays_clean, w4  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 272])
@pytest.mark.parametrize("e,eps", [(59, 1e-6), (70, 1e-6), (100, 1e-6), (126, 1e-6), (-60, 0.0), (-100, 0.0), (-125, 0.0),
                                   (-45, 1e-30), (-60, 1e-30), (-90, 1e-38)])
def test_rope_norm_of_any_size(w4, cuda_device, e, eps, D):  # noqa: F811
    """Heads whose squares 32 bits do not hold, beside others in the same warp, and one with an infinity."""
    import torch

    x = _normals((9, 3, D), 21, torch.bfloat16, cuda_device).clamp(-1.9, 1.9)
    x[::2] *= 2.0 ** e
    x[4, 1, 7] = float("inf")
    weight, table = (1 + 0.1 * _normals((D,), 22)).to(cuda_device), w4.rope_table(16, 32, device=cuda_device)
    places = torch.arange(9, dtype=torch.int32, device=cuda_device)
    y = _np(w4.rope(x, places, table, norm=weight, eps=eps))
    with np.errstate(invalid="ignore"):
        ref, mag = oa.rope(oa.head_norm(_np(x), _np(weight), np.float32(eps)), _np(table), _np(places)[None].astype(int))
        bad = np.isnan(ref)
        assert np.array_equal(np.isnan(y), bad) and bad[4, 1].any() and bad.sum() <= 2
        assert (np.abs(y - ref) <= oa.norm_rope_tolerance(ref, mag, "bf16"))[~bad].all()


@pytest.mark.parametrize("form", [None, *FORMS])
def test_append_norms_heads_of_any_size(w4, cuda_device, form):  # noqa: F811
    """Queries and keys too large to be squared in 32 bits, values as large that no norm touches."""
    r = Rows(w4, cuda_device, "bf16", form, 5, 2, 128, 16, [(1, 1), (20, 33), (9, 9)], seed=23)
    r.fused[::3] *= 2.0 ** 90
    weight = (1 + 0.1 * _normals((128,), 24)).to(cuda_device)
    for norms in (dict(q_norm=weight, k_norm=weight), dict(k_norm=weight), dict(q_norm=weight)):
        q = r.append(q=r.q, **norms)
        for x, normed, got in ((r.q, "q_norm" in norms, _np(q)), (r.k, "k_norm" in norms, None), (r.v, False, None)):
            ref = oa.head_norm(_np(x), _np(weight), np.float32(1e-6)) if normed else _np(x)
            off = 2 * oa.NORM * np.abs(ref) if normed else 0.0
            if got is not None:
                tol = oa.UNIT["bf16"] * np.abs(ref) + off + oa.TINY["bf16"]
            else:
                cache, scale = (r.k_cache, r.ks) if x is r.k else (r.v_cache, r.vs)
                got, _ = r.stored(cache, scale)
                tol = oa.held_tolerance(ref, form, off)[0] if form else oa.UNIT["bf16"] * np.abs(ref) + off
            assert (np.abs(got - ref) <= tol).all()


def test_heads_are_worked_on_once_in_place(w4, cuda_device):  # noqa: F811
    """Heads that share a thread with one too large to be squared, written over themselves: results whose squares are
    too small in turn (weights of 2^-50, no eps) are not taken for rows."""
    import torch

    x = _normals((20000, 8, 64), 25, torch.bfloat16, cuda_device)
    x[::3, 1::2] *= 2.0 ** 70
    weight = _normals((64,), 26).to(cuda_device) * 2.0 ** -50
    table, places = w4.rope_table(4, 64, device=cuda_device), torch.zeros(20000, dtype=torch.int32, device=cuda_device)
    apart = w4.rope(x, places, table, norm=weight, eps=0.0)
    w4.rope(x, places, table, norm=weight, eps=0.0, out=x)
    assert torch.equal(x, apart)
