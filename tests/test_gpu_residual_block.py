"""A residual block's operators together, as examples/residual_block.py runs them (GPU).

Each gradient against its formula in fp64 on the values that the step itself kept (the checkpoints' restored values,
the norms' factors) and computes from them.  Between the operators dr, dx, da, h and dh are bf16 and products are
within 1e-5 of their terms, so gradients are compared as vectors: dx is rounded once (2^-8 at most), dWdown once more,
da and dh each once more, h once; in all at most five roundings, 5 2^-8 of the gradient's norm, for the longest chain.
"""

import importlib.util
import os

import numpy as np
import pytest
import torch

from _util import f64
from layer_optimizer_gb300 import native, synth
from oracle import checkpoint as oc
from oracle import sandwich as osw

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("residual_block", os.path.join(ROOT, "examples", "residual_block.py"))
residual_block = importlib.util.module_from_spec(spec)
spec.loader.exec_module(residual_block)


def _restored(ck):
    q, scale = ck.tensors
    return oc.restore(f64(q.float()), f64(scale.float()), ck.group)


def _near(name, got, want, roundings):
    off = np.linalg.norm(f64(got.float()) - want) / np.linalg.norm(want)
    assert off <= roundings * 2.0 ** -8, (name, off)


@pytest.mark.parametrize("sequences,tokens,hidden,ffn,group", [(3, 65, 264, 528, 128), (2, 400, 1024, 512, 32), (1, 7, 64, 80, 0)])
def test_step_against_fp64(sequences, tokens, hidden, ffn, group):
    b = residual_block.ResidualBlock(sequences, tokens, hidden, ffn, group=group, seed=3)
    rows = sequences * tokens
    for i, k in enumerate(("g_in", "g_post", "g_pre")):
        b.weights[k].copy_((1.0 + synth.normal((hidden,), 0.2, 5 + i)).to(torch.bfloat16))
    r, dh, ds = (synth.normal((rows, hidden), std, 8 + i).to(torch.bfloat16).cuda() for i, std in enumerate((1.5, 1.0, 1.0)))
    s, h_next = b.forward(r)
    dr = b.backward(dh, ds)
    native.sf_sync_status()
    w = {k: f64(v.float()) for k, v in b.weights.items()}
    x, sr, rr, a = _restored(b.x8), _restored(b.s8), _restored(b.r8), _restored(b.a8)
    # forward: the checkpoints hold what the formulas give, within e4m3's half step and the bf16 values between
    f = osw.forward(f64(r.float()), None, None, w["g_in"], None, 0, 1.0, 1.0, 1e-5)
    u = np.maximum(f["h"] @ w["up"].T, 0.0)
    assert np.linalg.norm(a - u) <= (2.0 ** -4 + 2.0 ** -6) * np.linalg.norm(u)
    assert np.linalg.norm(x - u @ w["down"].T) <= (2.0 ** -4 + 2.0 ** -6) * np.linalg.norm(u @ w["down"].T)
    assert np.linalg.norm(sr - f64(s.float())) <= (2.0 ** -4 + 2.0 ** -8) * np.linalg.norm(f64(s.float()))
    g = osw.backward(f64(dh.float()), f64(ds.float()), x, sr, w["g_post"], w["g_pre"], w["gate"], tokens, 1.0, 0.5, f64(b.rstd_post), f64(b.rstd_pre))
    _near("g_post", b.grads["g_post"], g["dg1"][0], 1.01)
    _near("g_pre", b.grads["g_pre"], g["dg2"][0], 1.01)
    _near("gate", b.grads["gate"], g["dgate"][0], 1.01)
    dx = g["dx"][0]
    _near("down", b.grads["down"], dx.T @ a, 2.1)
    da = (dx @ w["down"]) * (a != 0)
    h = rr * f64(b.rstd_in)[:, None] * w["g_in"]
    _near("up", b.grads["up"], da.T @ h, 4.1)
    g_in = osw.backward(da @ w["up"], g["dr"][0], rr, rr, None, w["g_in"], None, 0, 1.0, 1.0, None, f64(b.rstd_in))
    _near("g_in", b.grads["g_in"], g_in["dg2"][0], 4.1)
    _near("dr", dr, g_in["dx"][0], 5.1)


def test_steps_move_every_weight_and_give_the_same_bits_again():
    made = []
    for _ in range(2):
        b = residual_block.ResidualBlock(2, 64, 256, 384, seed=4)
        before = {k: m.clone() for k, m in b.masters.items()}
        r, dh, ds = (synth.normal((128, 256), 1.0, 11 + i).to(torch.bfloat16).cuda() for i in range(3))
        for _ in range(3):
            b.forward(r)
            b.backward(dh, ds)
            b.update(native.hparams(lr=1e-2))
        native.sf_sync_status()
        assert all(torch.isfinite(m).all() and not torch.equal(m, before[k]) for k, m in b.masters.items())
        made.append(b.masters)
    assert all(torch.equal(made[0][k], made[1][k]) for k in made[0])


def test_main_runs(capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["residual_block", "--sequences", "2", "--tokens", "128", "--hidden", "256", "--ffn", "512", "--steps", "2"])
    residual_block.main()
    assert "MiB of activations kept" in capsys.readouterr().out
