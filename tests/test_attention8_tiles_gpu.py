"""The tiled kernel over an 8-bit cache where its two halves share a tile's blocks, on work lists whose order makes one
half wait for the other at the end of a tile while that one is already in the next. (Heads of 128 have a ring of a
block and a half, heads of 64 one of three and a half.)"""
import numpy as np
import pytest

from test_attention8_gpu import Batch8
from test_kv_cache8_gpu import FORMS
from test_paged_attention_gpu import DTYPES, w4  # noqa: F401
from test_paged_attention_tiles_gpu import _mixed_lens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("blocks", [5, 9])
def test_halves_that_wait_for_each_other(w4, cuda_device, blocks, D, form, dtype):  # noqa: F811
    """One cached head of 64 query heads: 1 or 2 tokens fill half a tile, and neighbouring tiles have different numbers
    of blocks. The calls must end without a wait that gives up, with the same bits whatever the timing."""
    lens = [(1 + n % 2, max(m, 2)) for n, m in _mixed_lens(np.random.default_rng(100 * blocks + D), blocks)]
    b = Batch8(cuda_device, dtype, form, 64, 1, D, 64, lens, seed=D)
    first, lse = b.attend(w4, return_lse=True)
    assert w4.device_status(raise_on_error=False) == 0
    for _ in range(30):
        assert (b.attend(w4) == first).all()
    assert w4.device_status(raise_on_error=False) == 0
    if form == "int8":  # (the formats differ in how bytes become fp16 alone)
        b.check(first, lse)
