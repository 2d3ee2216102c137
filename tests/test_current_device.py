"""Calls on tensors of a device that is not the current one are refused before
anything is launched (no GPU: the current device is a stand-in)."""
import pytest
import torch


@pytest.fixture()
def w4(monkeypatch):
    import w4a16_group_quantized_linear_gb300 as w4

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 64)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: type("Stream", (), {"cuda_stream": 64})())
    return w4


def test_another_device_is_refused(w4):
    with pytest.raises(ValueError, match="cuda:0"):
        w4._raw_stream(0)
    with pytest.raises(ValueError, match="cuda:0"):
        w4._stream(torch.device("cuda", 0))


def test_the_current_device_is_served(w4):
    assert w4._raw_stream(1) == 64
    assert w4._stream(torch.device("cuda", 1)).value == 64
    assert w4._stream(torch.device("cuda")).value == 64
