"""The binding's choice of stream (CPU: torch's stream calls are faked)."""
import importlib.util
import os
from types import SimpleNamespace

import pytest
import torch

import conftest

PKG = os.path.join(conftest.ROOT, "long_context_decode_indexpool_b200", "__init__.py")


def _fresh():
    conftest.build_lib()
    spec = importlib.util.spec_from_file_location("_spx_fresh", PKG)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("gone", [("_cuda_getCurrentRawStream",), ("_cuda_getDevice",),
                                  ("_cuda_getCurrentRawStream", "_cuda_getDevice")])
def test_stream_without_torch_s_private_calls(monkeypatch, gone):
    """A torch without the private calls still gives the current stream."""
    for name in gone:
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(cuda_stream=77))
    assert _fresh()._stream(None) == 77


def test_stream_of_the_current_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev, raising=False)
    m = _fresh()
    assert m._stream(None) == 103
    assert m._stream(5) == 5 and m._stream(SimpleNamespace(cuda_stream=9)) == 9


@pytest.mark.gpu
def test_stream_is_torch_s_current_one():
    from _gpu_helpers import need_gpu
    spx = need_gpu()
    assert spx._stream(None) == torch.cuda.current_stream().cuda_stream
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert spx._stream(None) == s.cuda_stream
    assert spx._stream(s) == s.cuda_stream
