"""What the Python layer keeps of its workspaces: a captured graph holds a
buffer's address, so no buffer that a graph may have seen is given back or
shared with calls outside the capture (no GPU: a stand-in for the library)."""
import ctypes
import gc
import weakref

import pytest
import torch


class FakeLibrary:
    """Zero-fills on the host and says which capture is under way."""

    def __init__(self):
        self.capture = 0
        self.zeroed = []

    def w4a16_workspace_init(self, ptr, nbytes, stream):
        ctypes.memset(ptr, 0, nbytes)
        self.zeroed.append((ptr.value, nbytes))
        return 0

    def w4a16_stream_capture_id(self, stream, out):
        out._obj.value = self.capture
        return 0


@pytest.fixture()
def kept(monkeypatch):
    import w4a16_group_quantized_linear_gb300 as w4

    fake = FakeLibrary()
    monkeypatch.setattr(w4, "_lib", fake)
    monkeypatch.setattr(w4, "_ws", {})
    for name, empty in (("_replaced", []), ("_captured", {})):
        if hasattr(w4, name):
            monkeypatch.setattr(w4, name, empty)
    cpu = torch.device("cpu")

    def get(nbytes, stream=64, kind="attention"):
        return w4._workspace(cpu, ctypes.c_void_p(stream), nbytes, kind)

    return get, fake


def test_a_replaced_workspace_stays_where_it_is(kept):
    get, fake = kept
    small = get(5 << 20)
    alive, at = weakref.ref(small), small.data_ptr()   # a graph captured now holds this address
    del small
    large = get(45 << 20)
    gc.collect()
    assert alive() is not None and alive().data_ptr() == at and large.data_ptr() != at
    # the larger one serves the small calls from then on, and nothing more is made
    assert get(5 << 20) is large and len(fake.zeroed) == 2


def test_many_sizes_keep_little(kept):
    get, _ = kept
    import w4a16_group_quantized_linear_gb300 as w4

    for n in range(2 << 20, 40 << 20, 1 << 20):
        last = get(n)
    assert sum(b.numel() for b in w4._replaced) <= last.numel() <= 2 * (39 << 20)


def test_a_first_call_under_capture_belongs_to_that_capture(kept):
    get, fake = kept
    fake.capture = 7
    one = get(5 << 20)
    assert get(4 << 20) is one and len(fake.zeroed) == 1     # one zero-fill in the graph
    larger = get(9 << 20)
    assert larger is not one and get(5 << 20) is larger
    fake.capture = 8                                          # another graph on the same stream
    two = get(5 << 20)
    assert two.data_ptr() != larger.data_ptr() and len(fake.zeroed) == 3
    fake.capture = 0                                          # and a call outside of both
    eager = get(5 << 20)
    assert eager is not two and len(fake.zeroed) == 4
    assert get(5 << 20) is eager


def test_a_stream_that_has_a_workspace_uses_it_under_capture(kept):
    """No zero-fill in the graph; one that has to be larger is the graph's."""
    get, fake = kept
    eager = get(5 << 20)
    fake.capture = 9
    assert get(5 << 20) is eager
    own = get(45 << 20)
    assert own is not eager and get(45 << 20) is own and get(5 << 20) is eager
    fake.capture = 0
    assert get(5 << 20) is eager and get(45 << 20) is not own


def test_streams_and_kinds_have_their_own(kept):
    get, _ = kept
    assert len({get(1 << 20, s, k).data_ptr() for s in (0, 64, 128) for k in ("linear", "attention")}) == 6


def test_capture_id_validation():
    from w4a16_group_quantized_linear_gb300 import build

    build.build()
    import w4a16_group_quantized_linear_gb300 as w4

    assert w4.lib().w4a16_stream_capture_id(None, None) == 1
