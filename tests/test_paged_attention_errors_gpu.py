"""The bounded waits of the tiled attention kernel, made to run out on purpose.

As in test_errors_gpu.py: in the test-hooks build a 1 ms limit and a loader
that stops after a few blocks make the waits give up; the kernel must record
W4A16_ERR_TIMEOUT, unwind, free its TMEM and return promptly, and the next
normal call must be correct. Nothing faults or hangs.
"""
import ctypes
import time

import pytest

from test_paged_attention_gpu import Batch

pytestmark = pytest.mark.gpu

TIMEOUT = 5
SHORT_NS, NORMAL_NS = 1_000_000, 2_000_000_000


@pytest.fixture()
def hooks(cuda_device, monkeypatch):
    import w4a16_group_quantized_linear_gb300 as w4
    from w4a16_group_quantized_linear_gb300 import build

    w4.lib()
    lib = ctypes.CDLL(build.build(variant="testhooks"))
    for name, (res, args) in w4.EXPORTS.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    lib.w4a16_test_set_hooks.restype = ctypes.c_int32
    lib.w4a16_test_set_hooks.argtypes = [ctypes.c_uint64, ctypes.c_int32]
    lib.w4a16_test_tmem_counters.restype = ctypes.c_int32
    lib.w4a16_test_tmem_counters.argtypes = [ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_uint64)]
    yield lib
    lib.w4a16_test_set_hooks(NORMAL_NS, -1)


def _tmem(lib):
    a, f = ctypes.c_uint64(0), ctypes.c_uint64(0)
    assert lib.w4a16_test_tmem_counters(ctypes.byref(a), ctypes.byref(f)) == 0
    return a.value, f.value


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,limits", [([(300, 4000)], (0, 1, 2, 3)), ([(40, 30000)], (0, 1, 2, 3)),
                                         ([(200, 200), (100, 700)], (0, 1))])   # a block for each SM at most
def test_wait_times_out_and_next_call_is_correct(hooks, cuda_device, lens, limits, D):
    import torch

    import w4a16_group_quantized_linear_gb300 as w4

    lib = hooks
    b = Batch(cuda_device, "fp16", 10, 2, D, 16, lens, seed=40)
    T = b.offsets[-1]
    c = w4._cache(b.k, b.v, b.page_table, b.q_offsets, b.kv_lens, b.q)
    out = torch.empty(T, 10, D, dtype=torch.float16, device=cuda_device)
    n = int(lib.w4a16_paged_attention_workspace_bytes(T, len(lens), 10, 2, D, b.max_q))
    ws = torch.empty(n, dtype=torch.uint8, device=cuda_device)
    st = w4._stream(cuda_device)

    def call():
        assert lib.w4a16_workspace_init(w4._ptr(ws), n, st) == 0
        return lib.w4a16_paged_attention(ctypes.byref(c), T, w4._ptr(b.q), b.q.stride(0), b.q.stride(1), 10, b.max_q,
                                         1, 0, D ** -0.5, w4._ptr(out), None, w4._ptr(ws), n, st)

    for issue_limit in limits:   # nothing; k; k and v; the next k
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
