"""The fp64 oracle of a residual block's end and its 8-bit checkpoints, pinned (CPU)."""

import numpy as np
import pytest
import torch

from oracle import checkpoint as oc
from oracle import norm as on
from oracle import sandwich as osw

EPS = 1e-5


def _case(seed, rows=7, cols=11, gates=3, post=True):
    rng = np.random.default_rng(seed)
    span = -(-rows // gates) if gates else 0
    v = dict(x=rng.standard_normal((rows, cols)), r=rng.standard_normal((rows, cols)),
             g1=1 + 0.2 * rng.standard_normal(cols) if post else None, g2=1 + 0.2 * rng.standard_normal(cols),
             gate=0.5 + 0.3 * rng.standard_normal((-(-rows // span), cols)) if gates else None)
    return v, span, rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols))


@pytest.mark.parametrize("gates,post", [(0, True), (1, True), (3, True), (7, True), (1, False), (4, False)])
def test_gradients_against_float64_autograd_and_differences(gates, post):
    v, span, dh, ds = _case(gates + 10 * post, gates=gates, post=post)
    a, b = 0.8, 0.3
    t = {k: None if u is None else torch.tensor(u, requires_grad=True) for k, u in v.items()}
    n = t["x"] if not post else t["x"] * torch.rsqrt(t["x"].square().mean(1, keepdim=True) + EPS) * t["g1"]
    at = torch.arange(len(dh)) // (span or len(dh))
    s = a * t["r"] + b * (n if not gates else t["gate"][at] * n)
    h = s * torch.rsqrt(s.square().mean(1, keepdim=True) + EPS) * t["g2"]
    ((h * torch.tensor(dh)).sum() + (s * torch.tensor(ds)).sum()).backward()
    f = osw.forward(v["x"], v["r"], v["g1"], v["g2"], v["gate"], span, a, b, EPS)
    assert np.allclose(f["s"], s.detach().numpy(), atol=1e-14) and np.allclose(f["h"], h.detach().numpy(), atol=1e-14)
    got = osw.backward(dh, ds, v["x"], f["s"], v["g1"], v["g2"], v["gate"], span, a, b, f["rho1"], f["rho2"])
    names = dict(dr="r", dx="x", dg1="g1", dg2="g2", dgate="gate")
    assert set(got) == {k for k, u in names.items() if v[u] is not None}
    loss = lambda w: (lambda o: (o["h"] * dh).sum() + (o["s"] * ds).sum())(  # noqa: E731
        osw.forward(w["x"], w["r"], w["g1"], w["g2"], w["gate"], span, a, b, EPS))
    rng = np.random.default_rng(5)
    for k, (g, mag) in got.items():
        assert np.allclose(g, t[names[k]].grad.numpy(), atol=1e-13)
        assert np.all(np.abs(g) <= mag * (1 + 1e-12))
        step = rng.standard_normal(g.shape)
        ends = [loss(dict(v, **{names[k]: v[names[k]] + e * step})) for e in (1e-5, -1e-5)]
        assert abs((ends[0] - ends[1]) / 2e-5 - (g * step).sum()) <= 1e-7 * (1 + np.abs(g * step).sum())


def test_one_gate_row_is_a_gate_of_every_row():
    v, span, dh, ds = _case(3, gates=1)
    f1 = osw.forward(v["x"], v["r"], v["g1"], v["g2"], v["gate"], 0, 1.0, 1.0, EPS)
    f2 = osw.forward(v["x"], v["r"], v["g1"], v["g2"], np.repeat(v["gate"], 7, axis=0), 1, 1.0, 1.0, EPS)
    assert np.array_equal(f1["h"], f2["h"])


@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_checkpoints_by_brute_force(group):
    rng = np.random.default_rng(group)
    v = rng.standard_normal((5, 70)) * np.exp(8 * rng.standard_normal((5, 1)))
    v[1, 3], v[1, 40], v[2], v[3, 5] = np.nan, -np.inf, 0.0, 2.0 ** -140
    v[4, :32] = 448.0 * 2.0 ** -3          # exactly at the largest value
    q, s = oc.quantize(v, group)
    codes = np.array([0.0] + [m * 2.0 ** -9 for m in range(1, 8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])
    assert codes[-1] == 448.0 and len(codes) == 127
    width = group or 70
    for i in range(5):
        for j in range(70):
            k = s[i, j // width]
            if not np.isfinite(v[i, j]):
                assert np.isnan(q[i, j])
                continue
            block = v[i, j // width * width:(j // width + 1) * width]
            top = np.abs(block[np.isfinite(block)]).max()
            assert top <= 448 * k and (top > 224 * k or k == 2.0 ** -126) and np.log2(k) == int(np.log2(k))
            assert abs(abs(q[i, j]) * k - abs(v[i, j])) == np.abs(codes * k - abs(v[i, j])).min()
            assert abs(q[i, j]) in codes
    assert np.array_equal(oc.restore(q, s, group), oc.spread(s, group, 70) * q, equal_nan=True)


def test_ties_go_to_the_even_code():
    assert np.array_equal(on.e4m3(np.array([17 / 16, 19 / 16, 2.0 ** -10, 3 * 2.0 ** -10])), [1.0, 1.25, 0.0, 2 * 2.0 ** -9])
