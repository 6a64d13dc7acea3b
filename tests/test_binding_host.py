"""What the binding asks torch for, without a GPU: the current stream."""
import sys
from types import SimpleNamespace

import pytest

from masking_tm_affine_gb300 import tm


def fake_torch(initialized=True, **private):
    cuda = SimpleNamespace(is_initialized=lambda: initialized, current_stream=lambda: SimpleNamespace(cuda_stream=0x77))
    return SimpleNamespace(cuda=cuda, _C=SimpleNamespace(**private))


@pytest.mark.parametrize("private,want", [
    (dict(_cuda_getCurrentRawStream=lambda d: 0x50 + d, _cuda_getDevice=lambda: 3), 0x53),
    (dict(), 0x77), (dict(_cuda_getCurrentRawStream=lambda d: 1), 0x77), (dict(_cuda_getDevice=lambda: 0), 0x77)])
def test_current_stream_with_and_without_private_functions(monkeypatch, private, want):
    monkeypatch.setitem(sys.modules, "torch", fake_torch(**private))
    assert tm._stream(None) == want


def test_streams_given_and_none(monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", fake_torch(initialized=False))
    assert tm._stream(None) is None                              # torch has no context yet: the default stream
    monkeypatch.delitem(sys.modules, "torch")
    assert tm._stream(None) is None and tm._stream(0x1234) == 0x1234
    assert tm._stream(SimpleNamespace(cuda_stream=0x99)) == 0x99
