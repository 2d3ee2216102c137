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
