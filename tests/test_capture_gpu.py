"""Captured graphs beside other calls on the stream that they were captured on."""
import numpy as np
import pytest

import workloads
from helpers import to_dev
from test_paged_attention_gpu import Batch

pytestmark = pytest.mark.gpu

STEP = [(1, 3000), (1, 700), (1, 1300)]      # divided between thread blocks: joined through the workspace
CHUNK = [(400, 900), (1, 50)]


@pytest.fixture(autouse=True)
def _fresh_workspaces(w4, cuda_device, monkeypatch):
    monkeypatch.setattr(w4, "_ws", {})
    yield
    assert w4.device_status(raise_on_error=False) == 0


@pytest.fixture(scope="module")
def w4():
    import w4a16_group_quantized_linear_gb300 as w4

    w4.lib()
    return w4


def _fill(dev, stream, value):
    """Takes what memory the allocator has free for this stream, in the sizes of the workspaces."""
    import torch

    with torch.cuda.stream(stream):
        return [torch.full((n << 20,), value, dtype=torch.uint8, device=dev) for n in (1, 2, 5, 6, 12, 26, 46) * 3]


@pytest.mark.parametrize("D", [64, 128])
def test_decode_graph_after_a_prompt_on_its_stream(w4, cuda_device, D):
    import torch

    step = Batch(cuda_device, "fp16", 10, 2, D, 16, STEP, seed=D)
    chunk = Batch(cuda_device, "fp16", 10, 2, D, 16, CHUNK, seed=D + 1)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        first = w4.paged_attention(*step.args(), 1).clone()
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            out = w4.paged_attention(*step.args(), 1)
        chunked = w4.paged_attention(*chunk.args(), chunk.max_q)   # needs a larger workspace
        s.synchronize()
    held = _fill(cuda_device, s, 0x55)
    torch.cuda.synchronize()
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    assert all(bool((t == 0x55).all()) for t in held)
    step.check(out)
    chunk.check(chunked)
    with torch.cuda.stream(s):
        assert torch.equal(w4.paged_attention(*chunk.args(), chunk.max_q), chunked)


def test_first_calls_under_capture(w4, cuda_device):
    """Two graphs on one stream that was never called on; the second one is replayed first, and the
    calls outside of the graphs come before either."""
    import torch

    a = Batch(cuda_device, "fp16", 10, 2, 128, 16, STEP, seed=3)
    b = Batch(cuda_device, "bf16", 10, 2, 64, 16, CHUNK, seed=4)
    s, ga, gb = torch.cuda.Stream(), torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(ga, stream=s):
        out_a = [w4.paged_attention(*a.args(), 1) for _ in range(3)]
    with torch.cuda.graph(gb, stream=s):
        out_b = [w4.paged_attention(*b.args(), b.max_q), w4.paged_attention(*b.args(), b.max_q)]
    with torch.cuda.stream(s):
        a.check(w4.paged_attention(*a.args(), 1))
        s.synchronize()
    for _ in range(2):
        gb.replay()
        ga.replay()
    torch.cuda.synchronize()
    for o in out_a:
        a.check(o)
    for o in out_b:
        b.check(o)
    # at the same time on two streams: each has a workspace of its own
    p, q = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(p):
            ga.replay()
        with torch.cuda.stream(q):
            gb.replay()
    torch.cuda.synchronize()
    for o in out_a:
        a.check(o)
    for o in out_b:
        b.check(o)


def test_linear_graph_after_a_larger_layer_on_its_stream(w4, cuda_device):
    """The layer's own workspace (group 64: partial sums in global memory)."""
    import torch

    def layer(N, K, seed):
        r = workloads.rng(seed)
        qw, sc = workloads.raw_packed(r, N, K, 64)
        return [to_dev(t, cuda_device) for t in (workloads.activations(r, 1, K), qw, sc)]

    small, large = layer(512, 4096, 1), layer(32768, 1024, 2)
    sizes = [w4.workspace_bytes(1, x[1].shape[0], x[0].shape[1], 64) for x in (small, large)]
    assert sizes[0] > 0
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        first = w4.linear(*small, 64).clone()
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            out = w4.linear(*small, 64)
        w4._workspace(cuda_device, w4._stream(cuda_device), 40 << 20)   # as a much larger problem would ask for
        w4.linear(*large, 64)
        s.synchronize()
    held = _fill(cuda_device, s, 0x55)
    torch.cuda.synchronize()
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    assert all(bool((t == 0x55).all()) for t in held)
    assert np.isfinite(first.float().cpu().numpy()).all()
