"""Which stream a call without one runs on (CPU only: a recording stand-in takes the library's place)."""

import pytest
import torch

from layer_optimizer_gb300 import native

HANDLE = 0xABCD0


class _Recorder:
    """Takes every call of the library and keeps its arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def recorder(monkeypatch):
    r = _Recorder()
    monkeypatch.setattr(native, "load", lambda path=None: r)
    return r


class _Stream:
    cuda_stream = HANDLE


@pytest.fixture
def side_stream(monkeypatch):
    """As under `with torch.cuda.stream(side)`."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _Stream())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: HANDLE, raising=False)


def _calls():
    m = native.sf_matrix(1 << 20, 4, 8, 8, native.SF_BF16)
    hp = native.hparams()
    P = type("P", (), {"handle": 4096})
    return {
        "sf_dropout": lambda **k: native.sf_dropout(m, m, 0.0, **k),
        "sf_add_rmsnorm_forward": lambda **k: native.sf_add_rmsnorm_forward(m, None, 4096, 1e-5, h=m, gain_dtype=0, **k),
        "sf_add_rmsnorm_backward": lambda **k: native.sf_add_rmsnorm_backward(m, m, 4096, 4096, dx=m, gain_dtype=0, **k),
        "lce_vocab_forward_backward": lambda **k: native.lce_vocab_forward_backward(m, m, 4096, **k),
        "lce_forward_backward": lambda **k: native.lce_forward_backward(1, 1, 1, 8, 8, 8, 8, -100, 1, 1, 1, 1, 1, **k),
        "sf_adamw_layer_step": lambda **k: native.sf_adamw_layer_step([(16, 16, 16, 16, None, 8)], hp, 1, **k),
        "sf_gemm_bf16": lambda **k: native.sf_gemm_bf16(1, 0, 1, 0, 1, 8, 8, 8, 8, 8, 8, **k),
        "lsp_compress": lambda **k: native.lsp_compress(P, P, 1, 0, 8, 8, 1, 1, 1, **k),
        "lsp_adamw_compressed": lambda **k: native.lsp_adamw_compressed(1, 1, 1, 1, 8, hp, 1, **k),
        "lsp_decompress_apply": lambda **k: native.lsp_decompress_apply(P, P, 1, 1, 0, None, 8, 8, 1, 1, **k),
        "sf_sync_status": lambda **k: native.sf_sync_status(**k),
    }


@pytest.mark.parametrize("name", list(_calls()))
def test_without_a_stream_calls_run_on_the_current_one(recorder, side_stream, name):
    _calls()[name]()
    (called, args), = recorder.calls
    assert called == name and args[-1] == HANDLE
    # a stream that is given is taken: a torch stream, a handle, and 0 for the legacy default stream
    for given, want in ((_Stream(), HANDLE), (0x1230, 0x1230), (0, 0)):
        recorder.calls.clear()
        _calls()[name](stream=given)
        assert recorder.calls[0][1][-1] == want


@pytest.mark.parametrize("name", list(_calls()))
def test_before_the_first_gpu_call_the_default_stream_is_current(recorder, monkeypatch, name):
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: False)
    _calls()[name]()
    assert not recorder.calls[0][1][-1]


def test_torch_without_the_raw_handle(recorder, side_stream, monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    native.sf_sync_status()
    assert recorder.calls == [("sf_sync_status", (HANDLE,))]


def test_a_window_keeps_the_streams_it_is_given(recorder, side_stream):
    # it owns its three streams for its lifetime: None stays the default stream, not whichever was current
    native.sf_window_create([[(16, 16, 16, 16, None, 8)]], None, 0x10, _Stream())
    name, args = recorder.calls[0]
    assert name == "sf_window_create" and not args[3] and args[4] == 0x10 and args[5] == HANDLE
