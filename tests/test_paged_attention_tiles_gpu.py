"""The tiled attention kernel where its two halves share a tile's blocks, on work lists whose order
makes one half wait for the other at the end of a tile while that one is already in the next.
"""
import numpy as np
import pytest

from test_paged_attention_gpu import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import w4a16_group_quantized_linear_gb300 as w4

    w4.lib()
    return w4


def _mixed_lens(r, blocks):
    """Sequences of 1 to 4 tokens whose tiles have mostly 1, 2 or 3 blocks of 128 places, in runs of
    `blocks` blocks and more for each SM, with a long one here and there that is divided between SMs."""
    lens, total = [], 0
    while total < blocks * 152:
        n = int(r.integers(1, 5))
        k = int(r.choice([1, 1, 1, 2, 2, 3, 4, 12]))
        lens.append((n, int(max(n, (k - 1) * 128 + r.integers(1, 129)))))
        total += k
    return lens


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("blocks", [5, 9, 16])
def test_halves_that_wait_for_each_other(w4, cuda_device, blocks, D):
    """One cached head: neighbouring tiles have different numbers of blocks. The calls must end without
    a wait that gives up, give the oracle's results, and the same bits whatever the timing."""
    b = Batch(cuda_device, "fp16", 32, 1, D, 64, _mixed_lens(np.random.default_rng(100 * blocks + D), blocks), seed=D)
    first, lse = w4.paged_attention(*b.args(), b.max_q, return_lse=True)
    assert w4.device_status(raise_on_error=False) == 0
    b.check(first, lse)
    for _ in range(30):
        again = w4.paged_attention(*b.args(), b.max_q)
        assert (again == first).all()
    assert w4.device_status(raise_on_error=False) == 0
