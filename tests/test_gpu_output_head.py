"""The output end's operators together, as examples/output_head.py runs them (GPU).

The whole step against fp64 written out here: norm, dropout, cross-entropy and
their gradients from the same bf16 inputs.  Between the operators h and dh are
bf16, so the gradients are compared as vectors: each of h, dZ, dh and the
results is rounded to bf16 at a relative error of at most 2^-8, in all less
than 2^-6 of the gradient's norm.
"""

import importlib.util
import os

import numpy as np
import pytest
import torch

from _util import f64
from layer_optimizer_gb300 import native, synth
from oracle import dropout as od
from oracle import norm as on
from oracle.lce import lce

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("output_head", os.path.join(ROOT, "examples", "output_head.py"))
output_head = importlib.util.module_from_spec(spec)
spec.loader.exec_module(output_head)


def _inputs(N, D, V, seed):
    x, r = synth.normal((N, D), 1.0, seed, dtype=torch.bfloat16), synth.normal((N, D), 1.5, seed + 1, dtype=torch.bfloat16)
    y = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    y[: N // 4] = -100
    return x.to(DEV), r.to(DEV), y.to(DEV)


def test_step_against_fp64():
    N, D, V = 190, 264, 1003
    head = output_head.OutputHead(N, D, V, p=0.25, seed=5, checkpoint=True)
    head.weights[0].copy_(1.0 + synth.normal((D,), 0.2, 9).to(DEV))
    x, r, y = _inputs(N, D, V, 3)
    loss = head.forward_backward(x, r, y, 77)
    native.sf_sync_status()
    gain, W = f64(head.weights[0].float()), f64(head.weights[1].float())
    s, _ = od.dropout(f64(x.float()), 0.25, 5, 77, f64(r.float()))
    h, _ = on.forward(s, gain, head.eps)
    ref = lce(h, W, y.cpu().numpy())
    ds, dg, _, _ = on.backward(ref["dH"], s, gain, head.eps)
    dx = np.where(od.mask(N, D, 0.25, 5, 77), ds * od.factor(0.25), 0.0)
    assert abs(float(loss) - ref["loss"]) <= 2.0 ** -8 * np.abs(ref["Z"]).max()
    for name, got, want in (("dW", head.grads[1], ref["dW"]), ("dgain", head.grads[0], dg), ("dr", head.dr, ds), ("dx", head.dx, dx)):
        got = f64(got.float())
        assert np.linalg.norm(got - want) <= 2.0 ** -6 * np.linalg.norm(want), name
    # the 8-bit copy of h stands for h within e4m3's half steps
    back = f64(head.h8.float()) * np.repeat(f64(head.h8_scale), 128, axis=1)[:, :D]
    assert np.all(np.abs(back - h) <= 2.0 ** -4 * np.abs(h) + 2.0 ** -9 * np.repeat(f64(head.h8_scale), 128, axis=1)[:, :D])


def test_step_gradients_against_differences():
    # the step's own loss at r + e d and r - e d: e is large against the bf16 rounding of h, small against its curvature
    N, D, V = 64, 128, 500
    head = output_head.OutputHead(N, D, V, p=0.1, seed=2)
    x, r, y = _inputs(N, D, V, 8)
    r = r.float().to(torch.bfloat16)
    head.forward_backward(x, r, y, 1)
    d = head.dr.float() / head.dr.float().norm()
    slope = float((head.dr.float() * d).sum())
    e = 4.0
    lo, hi = ((r.float() + k * d).to(torch.bfloat16) for k in (-e, e))
    up, down = float(head.forward_backward(x, hi, y, 1)), float(head.forward_backward(x, lo, y, 1))
    # h's bf16 rounding moves each token's loss by at most 2^-8 |h| |dz| in all; measured against the step along the gradient
    assert abs((up - down) / (2 * e) - slope) <= 0.1 * slope


def test_training_reduces_the_loss_and_repeats():
    N, D, V = 256, 256, 2000
    losses = []
    for _ in range(2):
        head = output_head.OutputHead(N, D, V, p=0.1, seed=4)
        x, r, y = _inputs(N, D, V, 6)
        hp = native.hparams(lr=1e-2)
        run = [head.step(x, r, y, hp).item() for _ in range(12)]
        native.sf_sync_status()
        assert run[0] == pytest.approx(np.log(V), rel=0.05) and run[-1] < 0.5 * run[0], run
        assert all(torch.equal(w, m.to(torch.bfloat16)) for w, m in zip(head.weights, head.masters))
        losses.append(run)
    assert losses[0] == losses[1]                       # the same bits on every run
