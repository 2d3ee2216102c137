"""Guard canaries of the attention operators: each writes exactly its outputs, and rows that a
call refuses stay as they were."""
import ctypes

import numpy as np
import pytest

from oracle import attention as oa
from test_paged_attention_gpu import Batch, _np, _t

pytestmark = pytest.mark.gpu

PATTERN = 12345
GUARD = 4096


@pytest.fixture(scope="module")
def w4():
    import w4a16_group_quantized_linear_gb300 as w4

    w4.lib()
    return w4


def _guarded(shape, dtype, dev):
    """A tensor between two stretches of guard elements."""
    import torch

    n = int(np.prod(shape))
    if dtype == torch.float32:
        buf = torch.full((n + 2 * GUARD,), PATTERN, dtype=torch.int32, device=dev)
    else:
        buf = torch.full((n + 2 * GUARD,), PATTERN, dtype=torch.int16, device=dev)
    return buf, buf[GUARD:GUARD + n].view(dtype).view(shape)


def _intact(buf):
    return bool((buf[:GUARD] == PATTERN).all()) and bool((buf[-GUARD:] == PATTERN).all())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[(1, 300), (1, 17)], [(3, 900), (1, 1)], [(20, 1500), (25, 25)],
                                  [(130, 400), (1, 9), (51, 3000)]])
def test_attention_writes_only_its_outputs(w4, cuda_device, lens, D, dtype):
    import torch

    b = Batch(cuda_device, dtype, 10, 2, D, 16, lens, seed=D)
    T = b.offsets[-1]
    buf, out = _guarded((T, 10, D), _t(dtype), cuda_device)
    lse_buf, lse = _guarded((T, 10), torch.float32, cuda_device)
    lib = w4.lib()
    n = int(lib.w4a16_paged_attention_workspace_bytes(T, len(lens), 10, 2, D, b.max_q))
    ws_buf = torch.full((n + 2 * GUARD,), 0x55, dtype=torch.uint8, device=cuda_device)
    ws, st = ws_buf[GUARD:GUARD + n], w4._stream(cuda_device)
    assert lib.w4a16_workspace_init(w4._ptr(ws), n, st) == 0
    c = w4._cache(b.k, b.v, b.page_table, b.q_offsets, b.kv_lens, b.q)
    k0, v0, q0 = b.k.clone(), b.v.clone(), b.fused.clone()
    for _ in range(2):
        assert lib.w4a16_paged_attention(ctypes.byref(c), T, w4._ptr(b.q), b.q.stride(0), b.q.stride(1), 10, b.max_q,
                                         1, 0, D ** -0.5, w4._ptr(out), w4._ptr(lse), w4._ptr(ws), n, st) == 0
    assert w4.device_status(raise_on_error=False) == 0
    b.check(out, lse)
    assert _intact(buf) and _intact(lse_buf)
    assert bool((ws_buf[:GUARD] == 0x55).all()) and bool((ws_buf[-GUARD:] == 0x55).all())
    assert torch.equal(b.fused, q0)
    assert torch.equal(b.k.view(torch.int16), k0.view(torch.int16))   # (NaN in them)
    assert torch.equal(b.v.view(torch.int16), v0.view(torch.int16))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,H,D,R", [(1, 5, 128, 128), (33, 3, 80, 64), (700, 22, 64, 64)])
def test_rope_writes_only_its_output(w4, cuda_device, T, H, D, R, dtype):
    import torch

    buf, out = _guarded((T, H + 1, D), _t(dtype), cuda_device)   # the last head is not this call's
    x = torch.randn(T, H, D, device=cuda_device).to(_t(dtype))
    table = w4.rope_table(64, R, device=cuda_device)
    pos = torch.arange(T, dtype=torch.int32, device=cuda_device) % 64
    w4.rope(x, pos, table, out=out[:, :H])
    assert w4.device_status(raise_on_error=False) == 0
    assert _intact(buf) and bool((out[:, H].view(torch.int16) == PATTERN).all())
    ref, mag = oa.rope(_np(x)[-1:], _np(table), _np(pos).astype(int)[None, -1:])
    assert (np.abs(_np(out[-1:, :H]) - ref) <= oa.rope_tolerance(ref, mag, dtype)).all()


@pytest.mark.parametrize("G,H", [(2, 10), (1, 1), (8, 40)])
def test_append_writes_only_its_outputs(w4, cuda_device, G, H):
    """q_out and the cache between guards; a cache whose heads are part of a wider row."""
    import torch

    lens = [(1, 20), (9, 40), (70, 70)]
    b = Batch(cuda_device, "fp16", H, G, 64, 16, lens, seed=H, poison=2.0)
    T, pages = b.offsets[-1], b.k.shape[0]
    bufs, caches = zip(*[_guarded((pages, 16, G + 1, 64), torch.float16, cuda_device) for _ in range(2)])
    k, v = (c[:, :, :G] for c in caches)
    k.copy_(b.k), v.copy_(b.v)
    k0, v0 = _np(k), _np(v)
    q_buf, q_out = _guarded((T, H, 64), torch.float16, cuda_device)
    kn, vn = (torch.randn(T, G, 64, device=cuda_device).half() for _ in range(2))
    w4.kv_append(kn, vn, k, v, b.page_table, b.q_offsets, b.kv_lens, q=b.q, q_out=q_out)
    assert w4.device_status(raise_on_error=False) == 0
    assert all(_intact(x) for x in (*bufs, q_buf)) and torch.equal(q_out, b.q)
    assert all(bool((c[:, :, G].contiguous().view(torch.int16) == PATTERN).all()) for c in caches)
    where = (b.table, b.offsets, b.kv)
    assert np.array_equal(_np(k), oa.append(k0, _np(kn), *where))
    assert np.array_equal(_np(v), oa.append(v0, _np(vn), *where))


@pytest.mark.parametrize("small", [1, 3, 49])
def test_rows_of_a_sequence_longer_than_max_q_len_are_not_written(w4, cuda_device, small):
    """Reported; the other sequences' rows are within the oracle's bounds."""
    import torch

    b = Batch(cuda_device, "fp16", 10, 2, 128, 16, [(50, 100), (1, 40), (1, 300)], seed=27)
    out = torch.full((52, 10, 128), 7.0, dtype=torch.float16, device=cuda_device)
    w4.paged_attention(*b.args(), small, out=out)
    assert w4.device_status(raise_on_error=False) == 6
    assert bool((out[:50] == 7.0).all())
    good = w4.paged_attention(*b.args(), 50)
    b.check(good)
    out[:50] = good[:50]
    b.check(out)
