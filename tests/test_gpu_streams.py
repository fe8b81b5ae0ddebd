"""Calls without a stream under torch.cuda.stream(side): they run on `side`, after what produces their inputs (GPU)."""

import pytest
import torch

from layer_optimizer_gb300 import native, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
SPIN = 50_000_000      # cycles: some 25 ms, far longer than a launch


def _late(*pairs):
    """On the current stream, some time from now: the first of each pair receives the second."""
    torch.cuda._sleep(SPIN)
    for dst, src in pairs:
        dst.copy_(src)


def _on_a_side_stream(make, inputs):
    """What make(inputs) gives when their values arrive late on a side stream, and when they are all there."""
    want = make(inputs)
    torch.cuda.synchronize()
    waiting = [torch.zeros_like(t) for t in inputs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _late(*zip(waiting, inputs))
        got = make(waiting)
        native.sf_sync_status()
        assert side.query(), "sf_sync_status waits for the current stream"
    for a, b in zip(got, want):
        assert torch.equal(a.float(), b.float())


def test_dropout_and_its_offset():
    x = synth.normal((64, 1024), 1.0, 1, dtype=BF).to(DEV)
    off = torch.tensor([77], device=DEV)

    def make(inputs):
        y = torch.empty_like(x)
        native.sf_dropout(inputs[0], y, 0.25, native.rng(3, 5, inputs[1]), residual=inputs[0])
        return [y]
    _on_a_side_stream(make, [x, off])


def test_norm_and_its_gradients():
    x, r = (synth.normal((200, 512), 1.0, s, dtype=BF).to(DEV) for s in (1, 2))
    gain = (1.0 + synth.normal((512,), 0.1, 3)).to(DEV)

    def make(inputs):
        x, r, gain = inputs
        s, h, dr = (torch.empty_like(x) for _ in range(3))
        rstd, dg = torch.empty(200, device=DEV), torch.empty(512, device=DEV)
        ws = torch.empty(native.sf_add_rmsnorm_workspace_bytes(200, 512), dtype=torch.uint8, device=DEV)
        native.sf_add_rmsnorm_forward(x, r, gain, 1e-5, sum=s, h=h, rstd=rstd)
        native.sf_add_rmsnorm_backward(h, s, gain, rstd, dresidual=dr, dgain=dg, ws=ws)
        return [s, h, rstd, dr, dg]
    _on_a_side_stream(make, [x, r, gain])


@pytest.mark.parametrize("N", [5, 100])
def test_cross_entropy_in_both_forms(N):
    D, V = 64, 600
    H, W = synth.normal((N, D), 1.0, 1, dtype=BF).to(DEV), synth.normal((V, D), 0.05, 2, dtype=BF).to(DEV)
    y = torch.arange(N, dtype=torch.int32, device=DEV)

    def vocab(inputs):
        loss, dH, dW = torch.empty(1, device=DEV), torch.empty_like(H), torch.empty_like(W)
        ws = torch.empty(native.lce_vocab_workspace_bytes(N, D, V), dtype=torch.uint8, device=DEV)
        native.lce_vocab_forward_backward(*inputs, loss=loss, dH=dH, dW=dW, ws=ws)
        return [loss, dH, dW]

    def chunks(inputs):
        loss, dH, dW = torch.empty(1, dtype=torch.float64, device=DEV), torch.empty(N, D, device=DEV), torch.empty(V, D, device=DEV)
        wsb = native.lce_workspace_bytes(N, D, V, 32)
        native.lce_forward_backward(*inputs, N, D, V, 32, -100, loss, dH, dW, torch.empty(wsb, dtype=torch.uint8, device=DEV), wsb)
        return [loss, dH, dW]
    for make in (vocab, chunks):
        _on_a_side_stream(make, [H, W, y])


def test_captured_without_naming_the_stream():
    # a capture's stream is the current one
    x = torch.ones(64, 512, device=DEV)
    y = torch.empty_like(x)
    native.sf_dropout(x, y, 0.5, native.rng(1, 0))
    want = y.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        native.sf_dropout(x, y, 0.5, native.rng(1, 0))
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
