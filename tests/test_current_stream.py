"""The stream that a call without one runs on, with and without torch's private
names."""
import sys
import types

import pytest

import moe_grouped_gemm_bf16_gb300 as dg


@pytest.mark.parametrize("private", [True, False])
def test_current_stream(monkeypatch, private):
    """With and without the private, faster lookups of torch."""
    torch = types.ModuleType("torch")
    torch._C = types.SimpleNamespace()
    stream = types.SimpleNamespace(cuda_stream=4096)
    torch.cuda = types.SimpleNamespace(is_initialized=lambda: True, current_stream=lambda: stream)
    if private:
        torch._C._cuda_getDevice = lambda: 3
        torch._C._cuda_getCurrentRawStream = lambda device: 4096 + device
    monkeypatch.setitem(sys.modules, "torch", torch)
    monkeypatch.setattr(dg, "_torch_stream", None)
    assert dg._stream(None) == (4099 if private else 4096)
    assert dg._stream(None) == (4099 if private else 4096)
    assert dg._stream(17) == 17 and dg._stream(stream) == 4096


def test_no_stream_before_torch_starts_cuda(monkeypatch):
    torch = types.ModuleType("torch")
    torch.cuda = types.SimpleNamespace(is_initialized=lambda: False)
    monkeypatch.setitem(sys.modules, "torch", torch)
    monkeypatch.setattr(dg, "_torch_stream", None)
    assert dg._stream(None) is None
    monkeypatch.delitem(sys.modules, "torch")
    assert dg._stream(None) is None
