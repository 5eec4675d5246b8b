"""The stream that a call of the binding takes by default: torch's current one, with or without torch's call for the raw handle."""

import sys
import types

import pytest

import hyper_connection_residual_hc_gb300 as hc


def _fake_torch(initialised, available, **c):
    cuda = types.SimpleNamespace(is_initialized=lambda: initialised, is_available=lambda: available,
                                 current_stream=lambda: types.SimpleNamespace(cuda_stream=77))
    return types.SimpleNamespace(cuda=cuda, _C=types.SimpleNamespace(**c))


def _default(monkeypatch, torch):
    for name in ("_torch", "_raw_stream", "_current_device"):
        monkeypatch.setattr(hc, name, None, raising=False)
    monkeypatch.setitem(sys.modules, "torch", torch)
    return hc._stream(None)


RAW = dict(_cuda_getCurrentRawStream=lambda device: 100 + device, _cuda_getDevice=lambda: 3)


def test_raw_handle_of_the_current_device(monkeypatch):
    assert _default(monkeypatch, _fake_torch(True, True, **RAW)) == 103


@pytest.mark.parametrize("has", [(), ("_cuda_getDevice",), ("_cuda_getCurrentRawStream",)])
def test_without_the_raw_handle(monkeypatch, has):
    assert _default(monkeypatch, _fake_torch(True, True, **{k: RAW[k] for k in has})) == 77


def test_before_torch_has_started_cuda(monkeypatch):
    assert _default(monkeypatch, _fake_torch(False, True, **RAW)) == 77
    assert _default(monkeypatch, _fake_torch(False, False)) is None


def test_a_given_stream_is_taken_as_it_is():
    assert hc._stream(5) == 5 and hc._stream(types.SimpleNamespace(cuda_stream=6)) == 6
