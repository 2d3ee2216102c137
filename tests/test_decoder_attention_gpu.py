"""The decoder attention example: prompts in chunks, then tokens from one
captured graph, against one chunk over each whole sequence.

The two ways round their queries, keys and values alike (the projections' kernels
differ by the number of rows, within 2^-9 of a value), so outputs agree to
a few roundings of fp16 (2^-11) of their largest value: 0.01 of it is allowed.
"""
import importlib.util
import os

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompts,steps,heads,kv_heads,head_dim", [
    ((37, 300, 5), 8, 16, 4, 64),
    ((1, 129), 1, 8, 8, 64),
    ((200, 16, 17, 128), 20, 10, 2, 128),
])
def test_growing_cache_gives_what_a_whole_chunk_gives(cuda_device, prompts, steps, heads, kv_heads, head_dim):
    path = os.path.join(ROOT, "examples", "decoder_attention.py")
    spec = importlib.util.spec_from_file_location("decoder_attention", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    grown, whole = example.run(prompts, steps, hidden=heads * head_dim // 128 * 128, heads=heads, kv_heads=kv_heads,
                               head_dim=head_dim)
    g, w = grown.float(), whole.float()
    assert g.isfinite().all() and w.abs().max() > 0
    assert (g - w).abs().max() <= 0.01 * w.abs().max()
