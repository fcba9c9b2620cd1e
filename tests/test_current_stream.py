"""Which stream an operator takes when none is given: torch's current one,
through whatever of its interfaces this torch has."""
import types

import pytest
import torch

import layer_streamed_gb300 as mt


@pytest.fixture
def fresh(monkeypatch):
    """A process that has made no call yet, on a device of our own."""
    monkeypatch.setattr(mt, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=0x77))
    return monkeypatch


def test_a_given_stream_is_taken_as_it_is(fresh):
    assert mt._stream(0) == 0 and mt._stream(0x1234) == 0x1234


@pytest.mark.parametrize("gone", [("_cuda_getCurrentRawStream",), ("_cuda_getDevice",),
                                  ("_cuda_getCurrentRawStream", "_cuda_getDevice")])
def test_a_torch_without_the_short_cut(fresh, gone):
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        fresh.setattr(torch._C, name, lambda *a: 0x55, raising=False)
    for name in gone:
        fresh.delattr(torch._C, name)
    assert mt._stream(None) == 0x77


def test_the_short_cut_asks_for_the_current_device(fresh):
    fresh.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    fresh.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0x100 + d, raising=False)
    assert mt._stream(None) == 0x103
    fresh.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    assert mt._stream(None) == 0x101  # asked anew at every call
