"""Host checks of the calls on an 8-bit cache and of the head norms (no GPU: they come
before any device work)."""
import ctypes

import pytest
import torch

from test_abi import _cache_struct, lib  # noqa: F401

P = 1 << 20


def _scales(**kw):
    import w4a16_group_quantized_linear_gb300 as w4

    return ctypes.byref(w4._CacheScales(**{**dict(format=1, k=P, v=P, page_stride=32, head_stride=16), **kw}))


def _norms(**kw):
    import w4a16_group_quantized_linear_gb300 as w4

    return ctypes.byref(w4._HeadNorms(**{**dict(q=P, k=P, eps=1e-6), **kw}))


SCALES = [(dict(format=0), 2), (dict(format=3), 2), (dict(k=None), 1), (dict(v=None), 1), (dict(k=P + 4), 3),
          (dict(v=P + 8), 3), (dict(page_stride=30), 1), (dict(head_stride=-16), 1), (dict(head_stride=6), 1)]
CACHES = [(dict(slot_stride=136), 1), (dict(head_stride=72), 1), (dict(page_stride=16 * 128 + 8), 1),
          (dict(dtype=3), 2), (dict(k=P + 8), 3), (dict(page_size=24), 2), (dict(head_dim=96), 2)]


@pytest.mark.parametrize("scales,cache,status", [(s, {}, e) for s, e in SCALES] + [({}, c, e) for c, e in CACHES])
def test_scales_and_caches(lib, scales, cache, status):  # noqa: F811
    c, s = ctypes.byref(_cache_struct(**cache)), _scales(**scales)
    assert lib.w4a16_kv_append_ex(c, s, 2, P, 128, 64, P, 128, 64, None, 0, 0, 0, None, None, None, None) == status
    assert lib.w4a16_kv_read(c, s, 2, P, P, None) == status
    assert lib.w4a16_paged_attention_ex(c, s, 2, P, 256, 64, 4, 1, 1, 0, 0.1, P, None, None, 0, None) == status


def test_nothing_to_do(lib):  # noqa: F811
    c = ctypes.byref(_cache_struct())
    s = _scales(k=None, v=None)
    assert lib.w4a16_kv_append_ex(c, s, 0, None, 128, 64, None, 128, 64, None, 0, 0, 0, None, None, None, None) == 0
    assert lib.w4a16_kv_read(c, s, 0, None, None, None) == 0
    assert lib.w4a16_paged_attention_ex(c, s, 0, None, 256, 64, 4, 1, 1, 0, 0.1, None, None, None, 0, None) == 0


def test_read(lib):  # noqa: F811
    c, s = ctypes.byref(_cache_struct()), _scales()
    assert lib.w4a16_kv_read(c, s, -1, P, P, None) == 1
    assert lib.w4a16_kv_read(c, s, 2, None, P, None) == 1 and lib.w4a16_kv_read(c, s, 2, P, None, None) == 1
    assert lib.w4a16_kv_read(c, s, 2, P + 8, P, None) == 3 and lib.w4a16_kv_read(c, None, 2, P, P + 2, None) == 3
    assert lib.w4a16_kv_read(None, s, 2, P, P, None) == 1


@pytest.mark.parametrize("norms,status", [(dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1),
                                          (dict(eps=float("inf")), 1), (dict(q=P + 4), 3), (dict(k=P + 8), 3)])
def test_norms(lib, norms, status):  # noqa: F811
    import w4a16_group_quantized_linear_gb300 as w4

    c = ctypes.byref(_cache_struct())
    for s in (None, _scales()):
        assert lib.w4a16_kv_append_ex(c, s, 2, P, 128, 64, P, 128, 64, P, 256, 64, 4, P, _norms(**norms), None,
                                      None) == status
    r = ctypes.byref(w4._Rotary(table=P, rows=8, rotary_dim=64, interleaved=0, positions=P, axes=1, pair_axes=None))
    n = {**dict(q=P, eps=1e-6), **norms}
    if "k" not in norms:
        assert lib.w4a16_rope_norm(1, P, 256, 64, P, 256, 64, 2, 4, 64, n["q"], n["eps"], r, None) == status


def test_rope_norm(lib):  # noqa: F811
    import w4a16_group_quantized_linear_gb300 as w4

    r = ctypes.byref(w4._Rotary(table=P, rows=8, rotary_dim=64, interleaved=0, positions=P, axes=1, pair_axes=None))
    assert lib.w4a16_rope_norm(1, P, 256, 64, P, 256, 64, 2, 4, 64, None, 1e-6, r, None) == 1
    assert lib.w4a16_rope_norm(1, P, 256, 64, P, 256, 64, 2, 4, 528, P, 1e-6, r, None) == 2
    assert lib.w4a16_rope_norm(1, P, 256, 64, P, 256, 64, 0, 4, 64, P, 1e-6, r, None) == 0
    assert lib.w4a16_rope_norm(1, P, 256, 64, P, 256, 64, 2, 4, 64, P, 1e-6, None, None) == 1


# --------------------------------------------------------- the Python layer --

def test_scales_belong_to_8_bit_caches():
    import w4a16_group_quantized_linear_gb300 as w4

    scale = torch.zeros(2, 3, 16)
    for cache in (torch.zeros(2, 16, 3, 64, dtype=torch.float16), torch.zeros(2, 16, 3, 64, dtype=torch.uint8)):
        assert w4._packed_scales(cache, None, None, -1) is None
        with pytest.raises(ValueError, match="8-bit cache's"):
            w4._packed_scales(cache, scale, scale, -1)
    for dtype in (torch.int8, torch.float8_e4m3fn):
        cache = torch.zeros(2, 16, 3, 64, dtype=torch.uint8).view(dtype)
        assert len(w4._packed_scales(cache, scale, scale.clone(), -1)) == ctypes.sizeof(w4._CacheScales)
        for k, v in ((None, None), (scale, None), (scale.double(), scale), (scale[0], scale[0])):
            with pytest.raises(ValueError, match="_scale: an 8-bit cache needs"):
                w4._packed_scales(cache, k, v, -1)
        with pytest.raises(ValueError, match="same shape"):
            w4._packed_scales(cache, scale, scale[:1], -1)
        other = torch.zeros(2, 16, 3)
        with pytest.raises(ValueError, match="pages, kv_heads, page_size"):
            w4._packed_scales(cache, other, other, -1)
        strided = torch.zeros(2, 3, 32)[:, :, ::2]
        with pytest.raises(ValueError, match="contiguous"):
            w4._packed_scales(cache, strided, strided, -1)


def test_norm_weights():
    import w4a16_group_quantized_linear_gb300 as w4

    assert w4._norm(None, "norm", 64, -1) == 0
    good = torch.ones(64)
    assert w4._norm(good, "norm", 64, -1) == good.data_ptr()
    for bad in (torch.ones(64).half(), torch.ones(32), torch.ones(1, 64), torch.ones(128)[::2], [1.0] * 64):
        with pytest.raises(ValueError, match="norm: expected"):
            w4._norm(bad, "norm", 64, -1)
