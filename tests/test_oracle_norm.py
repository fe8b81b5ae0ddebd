"""Pins of the dropout and norm oracles (CPU): published generator vectors, differences, closed forms, refusals."""

import ctypes

import numpy as np
import pytest
import torch

from layer_optimizer_gb300 import build, native
from oracle import dropout as od
from oracle import norm as on


@pytest.mark.parametrize("counter,key,want", [
    # the generator authors' known answers for philox4x32-10
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_generator_known_answers(counter, key, want):
    assert tuple(od.philox4x32(counter, key)) == want


def test_mask_follows_the_generator_word_by_word():
    rows, cols, seed, off = 3, 21, 0x123456789ABCDEF0, (7 << 32) + 5
    m = od.mask(rows, cols, 0.3, seed, off)
    for r in range(rows):
        for c in range(cols):
            b = r * 3 + c // 8
            w = od.philox4x32((b & od.LOW, b >> 32, off & od.LOW, off >> 32), (seed & od.LOW, seed >> 32))[(c % 8) // 2]
            bits = w & 0xFFFF if c % 2 == 0 else w >> 16
            assert m[r, c] == (bits >= od.threshold(0.3))


def test_mask_rate_and_expectation():
    m = od.mask(1000, 1000, 0.1, 99, 3)
    p = od.threshold(0.1) / 65536
    # binomial: 6 standard deviations of the mean of 10^6 draws
    assert abs(m.mean() - (1 - p)) < 6 * np.sqrt(p * (1 - p) / m.size)
    assert od.factor(0.1) * (1 - p) == pytest.approx(1.0, abs=1e-15)
    assert not od.mask(4, 9, 1.0, 1, 1).any() and od.factor(1.0) == 0.0


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(3)
    s, g, dh = rng.normal(size=(3, 7)), rng.normal(1.0, 0.2, size=7), rng.normal(size=(3, 7))
    eps = 1e-3
    ds, dg, _, _ = on.backward(dh, s, g, eps)

    def loss(s_, g_):
        return float((on.forward(s_, g_, eps)[0] * dh).sum())

    step = 1e-6
    for i in np.ndindex(*s.shape):
        d = np.zeros_like(s)
        d[i] = step
        # second-order differences: truncation ~ step^2, rounding ~ 1e-16 / step
        assert ds[i] == pytest.approx((loss(s + d, g) - loss(s - d, g)) / (2 * step), abs=1e-8)
    for j in range(7):
        d = np.zeros_like(g)
        d[j] = step
        assert dg[j] == pytest.approx((loss(s, g + d) - loss(s, g - d)) / (2 * step), abs=1e-8)


def test_norm_gradient_against_autograd_and_orthogonality():
    rng = np.random.default_rng(4)
    s, g, dh = rng.normal(size=(5, 16)), rng.normal(1.0, 0.2, size=16), rng.normal(size=(5, 16))
    S, G = (torch.tensor(v, requires_grad=True) for v in (s, g))
    h = S * torch.rsqrt((S * S).mean(dim=1, keepdim=True)) * G
    h.backward(torch.tensor(dh))
    ds, dg, _, _ = on.backward(dh, s, g, 0.0)
    assert np.allclose(ds, S.grad.numpy(), atol=1e-13) and np.allclose(dg, G.grad.numpy(), atol=1e-13)
    # without eps, h does not change along s, so the gradient is orthogonal to s
    assert np.abs((ds * s).sum(axis=1)).max() < 1e-13


def test_e4m3_rounding_against_every_code():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    vals = np.unique(codes[np.isfinite(codes)])
    assert vals.max() == 448.0
    assert np.array_equal(on.e4m3(vals), vals)
    mid = (vals[1:] + vals[:-1]) / 2
    lo, hi = on.e4m3(mid - 1e-9), on.e4m3(mid + 1e-9)
    assert np.array_equal(lo, vals[:-1]) and np.array_equal(hi, vals[1:])
    # ties go to the neighbour whose last fraction bit is 0, as torch rounds them
    assert np.array_equal(on.e4m3(mid), torch.tensor(mid).float().to(torch.float8_e4m3fn).double().numpy())


def test_quantize_zero_and_full_groups():
    h = np.zeros((2, 70))
    h[1, 64] = -3.5
    q, scale, each = on.quantize(h, 64)
    assert scale.shape == (2, 2) and scale[0, 0] == 2.0 ** -126 and scale[1, 1] == 3.5 / 448
    assert q[1, 64] == -448.0 and not q[0].any() and each.shape == h.shape


def _m(rows=4, cols=8, ld=None, dtype=native.SF_BF16, data=1 << 20):
    return native.sf_matrix(data, rows, cols, cols if ld is None else ld, dtype)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return native.load()


def test_dropout_refusals(lib):
    r = native.rng(1, 2)

    def call(x, res, y, p=0.1, g=r):
        return lib.sf_dropout(native._ref(x), native._ref(res), native._ref(y), p, native._ref(g), None)

    inv, uns = native.SF_ERR_INVALID, native.SF_ERR_UNSUPPORTED
    assert call(None, None, _m()) == inv
    assert call(_m(), None, None) == inv
    assert call(_m(), None, _m(rows=5)) == inv
    assert call(_m(), _m(cols=9), _m()) == inv
    assert call(_m(), _m(dtype=native.SF_FP32), _m()) == inv          # residual and y differ in type
    assert call(_m(ld=7), None, _m()) == inv
    assert call(_m(data=None), None, _m()) == inv
    assert call(_m(data=(1 << 20) + 1), None, _m()) == inv            # a bf16 matrix at an odd address
    assert call(_m(dtype=native.SF_E4M3), None, _m()) == uns
    assert call(_m(rows=-1), None, _m(rows=-1)) == inv
    for p in (-0.1, 1.5, float("nan")):
        assert call(_m(), None, _m(), p) == inv
    assert call(_m(), None, _m(), 0.1, None) == inv and "rng" in native.sf_last_error()
    assert call(_m(rows=0), None, _m(rows=0)) == native.SF_OK         # nothing to do
    assert call(_m(rows=1 << 40, ld=1 << 40), None, _m(rows=1 << 40, ld=1 << 40)) == uns


def test_norm_refusals(lib):
    inv, uns = native.SF_ERR_INVALID, native.SF_ERR_UNSUPPORTED

    def fwd(x=_m(), res=None, gain=1 << 20, gdt=native.SF_FP32, eps=1e-5, p=0.0, rng=None, s=None, h=_m(), q=None,
            scale=None, group=0):
        R = native._ref
        return lib.sf_add_rmsnorm_forward(R(x), R(res), gain, gdt, eps, p, R(rng), R(s), R(h), R(q), scale, group, None,
                                          None)

    assert fwd(x=None) == inv and fwd(gain=None) == inv and fwd(h=None) == inv
    assert fwd(gdt=native.SF_E4M3) == uns
    assert fwd(eps=-1.0) == inv and fwd(eps=float("nan")) == inv and fwd(eps=float("inf")) == inv
    assert fwd(h=_m(dtype=native.SF_FP32)) == inv                     # h has x's type
    assert fwd(res=_m(), s=_m(dtype=native.SF_FP32)) == inv           # sum has residual's type
    assert fwd(res=_m(rows=3)) == inv
    q = _m(dtype=native.SF_E4M3)
    assert fwd(q=q, scale=None) == inv and fwd(q=q, scale=1 << 20, group=16) == inv
    assert fwd(q=_m(), scale=1 << 20) == uns
    assert fwd(p=0.1) == inv                                          # no generator
    assert fwd(x=_m(cols=0), h=_m(cols=0)) == inv
    wide = 16385
    assert fwd(x=_m(cols=wide), h=_m(cols=wide)) == uns and "16384" in native.sf_last_error()
    assert fwd(x=_m(rows=0), h=_m(rows=0)) == native.SF_OK

    def bwd(dh=_m(), s=_m(), gain=1 << 20, rstd=1 << 20, dsum=None, dr=_m(), dx=None, dg=None, ws=None, wsb=0, p=0.0):
        R = native._ref
        return lib.sf_add_rmsnorm_backward(R(dh), R(s), gain, native.SF_FP32, rstd, R(dsum), p, None, R(dr), R(dx), dg,
                                           native.SF_FP32, ws, wsb, None)

    assert bwd(dh=None) == inv and bwd(s=None) == inv and bwd(gain=None) == inv and bwd(rstd=None) == inv
    assert bwd(dr=None) == inv and "all NULL" in native.sf_last_error()
    assert bwd(dsum=_m(dtype=native.SF_FP32)) == uns and bwd(dx=_m(dtype=native.SF_FP32)) == uns
    assert bwd(dg=1 << 20, ws=None) == inv and "workspace" in native.sf_last_error()
    assert bwd(dg=1 << 20, ws=1 << 20, wsb=4 * 8 * 4 - 1) == inv
    assert bwd(p=0.5) == inv
    assert native.sf_add_rmsnorm_workspace_bytes(4, 8) == 4 * 8 * 4
    assert native.sf_add_rmsnorm_workspace_bytes(0, 8) == 8 * 4
    assert native.sf_add_rmsnorm_workspace_bytes(4, 0) == 0


def test_binding_refuses_misfit_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(native.SfError, match="device or pinned"):
        native.matrix(x)
    with pytest.raises(native.SfError, match="two-dimensional"):
        native.matrix(x[0])
    with pytest.raises(native.SfError, match="unit column stride"):
        native.matrix(x.t())
    with pytest.raises(native.SfError, match="dense with 9"):
        native._vector(x[0], 9, "gain")
    with pytest.raises(native.SfError, match="not taken"):
        native._vector(x[0].double(), 8, "rstd", native._F32)
