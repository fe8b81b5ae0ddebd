"""Dropout with the residual's addition and the RMS norm against the fp64 oracle (GPU).

Tolerances, derived from the arithmetic (u = 2^-24, one fp32 rounding):

* y and s: the factor, its product and the addition round once each, so
  4u of the terms' magnitudes, plus half a unit in the output type's last
  place.
* rstd: a sum of positive squares, at most 32 in a row per thread and then
  at most 5 + 16 additions (48u), the squares' own error through s, a
  rounded mean, rsqrt within 2 ulp: half of it passes to rstd; 64u is taken.
* h: rstd's error, two products, s's error; then the output type's rounding.
* e4m3: half a quantum of the scaled value, plus the fp32 error of h / scale.
* ds: a sum of up to 16384 signed terms in chains of 32 + 21 (64u of the
  magnitudes), about ten more roundings: 96u of the terms' magnitudes.
* dgain: chains of at most rows / blocks + blocks / 32 + 5 additions; the
  cases here stay below 128: 160u of the magnitudes.
"""

import numpy as np
import pytest
import torch

from _util import f64
from layer_optimizer_gb300 import native, synth
from oracle import dropout as od
from oracle import norm as on

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
E4 = torch.float8_e4m3fn
EPS = 1e-5
SEED, OFF = 0x9E3779B97F4A7C15, (3 << 32) + 17


def _rows(rows, cols, pad, dtype, seed=None, std=1.0, lead=0):
    """A [rows, cols] view inside a wider, guarded buffer (lead extra elements in front, pad behind every row)."""
    buf = torch.full((lead + rows * (cols + pad) + 64,), 7.0, dtype=F32, device=DEV).to(dtype)
    v = buf[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    if seed is not None:
        v.copy_(synth.normal((rows, cols), std, seed).to(dtype))
    return v, buf


def _guard_ok(view, buf, lead=0):
    """Everything around the view still holds the fill."""
    rows, cols = view.shape
    b = buf.float().clone()
    b[lead:lead + rows * view.stride(0)].view(rows, -1)[:, :cols] = 7.0
    return bool((b == 7.0).all())


def _stored(dtype, ref, err):
    """Bound of a value known within err and stored in dtype: err plus half a unit in its last place (bf16 has 8
    significant bits, fp32 24)."""
    _, e = np.frexp(np.abs(ref) + err)
    return err + np.ldexp(0.5, e - (8 if dtype == BF else 24))


def _close(name, got, ref, bound):
    err = np.abs(f64(got.float()) - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(np.max(err / np.maximum(bound, 1e-300))))


SHAPES = [
    (1, 1, 0, 0), (1, 7, 0, 0), (3, 8, 0, 0), (2, 4096, 0, 0), (1, 16384, 0, 0), (5, 1000, 0, 0),
    (37, 1021, 0, 0),        # odd rows: unaligned from the second row on
    (300, 33, 7, 0),         # many short rows in a padded buffer
    (64, 256, 3, 0),         # a leading dimension off the unit
    (64, 256, 8, 1),         # a base off the unit
    (700, 128, 0, 0), (400, 2048, 16, 8), (161, 2056, 0, 0),
]


# rows that start at every place of a unit, several of them a thread in the backward pass
SHIFTED = [(2500, 1021, 0, 0), (5000, 61, 0, 0), (700, 4095, 0, 0), (620, 513, 5, 0), (400, 130, 1, 0), (40, 16375, 0, 0),
           (40, 16377, 0, 0), (700, 3, 0, 0), (500, 9, 0, 0), (333, 15, 2, 0)]


@pytest.mark.parametrize("rows,cols,pad,lead", SHAPES + SHIFTED)
@pytest.mark.parametrize("xt,yt,res,p", [(BF, BF, False, 0.1), (BF, F32, True, 0.5), (F32, BF, True, 0.01), (F32, F32, False, 0.25),
                                         (BF, BF, True, 0.0)])
def test_dropout_matches_oracle(rows, cols, pad, lead, xt, yt, res, p):
    x, _ = _rows(rows, cols, pad, xt, 1 + rows + cols, 1.0, lead)
    r, _ = _rows(rows, cols, pad, yt, 2 + rows + cols, 3.0, lead) if res else (None, None)
    y, buf = _rows(rows, cols, pad, yt, None, lead=lead)
    native.sf_dropout(x, y, p, native.rng(SEED, OFF) if p else None, residual=r)
    native.sf_sync_status()
    ref, mag = od.dropout(f64(x.float()), p, SEED, OFF, None if r is None else f64(r.float()))
    _close("y", y, ref, _stored(yt, ref, 4 * U * mag))
    assert _guard_ok(y, buf, lead)
    if p and not res:
        # the mask itself, exactly: dropped elements are 0 and kept ones are not (normal draws are never 0)
        kept = od.mask(rows, cols, p, SEED, OFF)
        assert np.array_equal(f64(y.float()) != 0, kept & (f64(x.float()) != 0))


def test_dropout_special_values_in_place_and_device_offset():
    rows, cols, p = 33, 40, 0.5
    x = torch.full((rows, cols), float("nan"), device=DEV)
    x[1::2] = float("inf")
    kept = od.mask(rows, cols, p, 5, 11)
    y = torch.empty_like(x)
    native.sf_dropout(x, y, p, native.rng(5, 11))
    got = f64(y)
    assert np.array_equal(got == 0, ~kept)               # a dropped NaN or infinity is 0
    assert np.isnan(got[0::2][kept[0::2]]).all() and np.isinf(got[1::2][kept[1::2]]).all()
    # everything dropped, nothing dropped
    native.sf_dropout(x, y, 1.0, native.rng(5, 11))
    assert not y.any()
    z = synth.normal((rows, cols), 1.0, 9).to(DEV)
    native.sf_dropout(z, y, 2.0 ** -18)
    assert torch.equal(y, z)
    # in place, and the offset split between host and device
    want = torch.empty_like(z)
    native.sf_dropout(z, want, p, native.rng(5, 11), residual=x.nan_to_num(1.0, 2.0))
    off = torch.tensor([4], device=DEV)
    w = z.clone()
    native.sf_dropout(w, w, p, native.rng(5, 7, off), residual=x.nan_to_num(1.0, 2.0))
    assert torch.equal(w, want)
    native.sf_sync_status()


def test_dropout_graph_replays_draw_new_masks():
    x = torch.ones(64, 512, device=DEV)
    y = torch.empty_like(x)
    off = torch.zeros(1, dtype=torch.int64, device=DEV)
    native.sf_dropout(x, y, 0.5, native.rng(1, 0, off))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        native.sf_dropout(x, y, 0.5, native.rng(1, 0, off), stream=torch.cuda.current_stream())
        off.add_(1)
    off.zero_()
    for step in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(f64(y) != 0, od.mask(64, 512, 0.5, 1, step))


def _forward_refs(x, r, gain, p, group):
    s, mag = od.dropout(f64(x.float()), p, SEED, OFF, None if r is None else f64(r.float()))
    h, rstd = on.forward(s, f64(gain.float()), EPS)
    # relative error of rstd: the squares' sum, and s's own error through it
    rel = 64 * U + 4 * U * np.mean(mag * np.abs(s), axis=1) * rstd ** 2
    eh = np.abs(h) * (rel + 4 * U)[:, None] + 4 * U * mag * rstd[:, None] * np.abs(f64(gain.float()))
    return s, mag, h, rstd, rel, eh


@pytest.mark.parametrize("rows,cols,pad,lead", SHAPES + SHIFTED)
@pytest.mark.parametrize("at,st,gt,res,p,group", [
    (BF, BF, BF, True, 0.0, None), (BF, F32, F32, True, 0.1, 128), (F32, F32, F32, True, 0.0, 0), (F32, BF, BF, True, 0.5, 32),
    (BF, BF, F32, False, 0.0, 64),
])
def test_add_rmsnorm_forward_matches_oracle(rows, cols, pad, lead, at, st, gt, res, p, group):
    x, _ = _rows(rows, cols, pad, at, 11 + rows + cols, 1.0, lead)
    r, _ = _rows(rows, cols, pad, st, 12 + rows + cols, 2.0, lead) if res else (None, None)
    gain = (1.0 + synth.normal((cols,), 0.2, 13 + cols)).to(gt).to(DEV)
    s, sbuf = _rows(rows, cols, pad, st, None, lead=lead)
    h, hbuf = _rows(rows, cols, pad, at, None, lead=lead)
    q = scale = qbuf = None
    if group is not None:
        q, qbuf = _rows(rows, cols, pad, E4, None, lead=lead)
        n = -(-cols // group) if group else 1
        scale = torch.full((rows, n), float("nan"), device=DEV)
    rstd = torch.full((rows,), float("nan"), device=DEV)
    native.sf_add_rmsnorm_forward(x, r, gain, EPS, sum=s, h=h, h8=q, h8_scale=scale, group=group or 0, rstd=rstd, p=p,
                                  rng=native.rng(SEED, OFF))
    native.sf_sync_status()
    rs, mag, rh, rr, rel, eh = _forward_refs(x, r, gain, p, group)
    _close("sum", s, rs, _stored(st, rs, 4 * U * mag))
    _close("rstd", rstd, rr, rel * rr)
    _close("h", h, rh, _stored(at, rh, eh))
    assert _guard_ok(s, sbuf, lead) and _guard_ok(h, hbuf, lead)
    if group is not None:
        assert _guard_ok(q, qbuf, lead)
        _, rsc, each = on.quantize(rh, group)
        width = group or cols
        esc = np.stack([eh[:, c:c + width].max(axis=1) for c in range(0, cols, width)], axis=1) / 448 + 4 * U * rsc
        _close("scale", scale, rsc, esc)
        got = f64(scale)
        sc = np.repeat(got, width, axis=1)[:, :cols]
        v = f64(q.float())
        assert np.abs(v).max() <= 448
        # h / scale within half a quantum of the stored value (the quantum of the larger of the two)
        quantum = on.e4m3_quantum(np.minimum(448.0, np.maximum(np.abs(v), np.abs(rh / sc))))
        assert np.all(np.abs(v - rh / sc) <= 0.5 * quantum + eh / sc + 4 * U * np.abs(rh / sc)), "e4m3"


def test_add_rmsnorm_forward_zero_rows_and_special_values():
    rows, cols = 6, 300
    x = synth.normal((rows, cols), 1.0, 3).to(DEV)
    x[0] = 0.0
    x[1, 250] = float("nan")
    x[2, 7] = float("inf")
    x[3] = 1e-30                                    # squares underflow: eps alone
    x[4] = 1e25                                     # squares overflow: rstd 0
    gain = torch.ones(cols, device=DEV)
    h, q = torch.empty_like(x), torch.empty(rows, cols, dtype=E4, device=DEV)
    scale, rstd = torch.empty(rows, 3, device=DEV), torch.empty(rows, device=DEV)
    native.sf_add_rmsnorm_forward(x, None, gain, EPS, h=h, h8=q, h8_scale=scale, group=128, rstd=rstd)
    native.sf_sync_status()
    assert not h[0].any() and not q[0].float().any() and torch.all(scale[0] == 2.0 ** -126)
    assert abs(float(rstd[0]) * EPS ** 0.5 - 1) < 1e-6
    assert torch.isnan(h[1]).all() and torch.isnan(q[1].float()).all() and torch.isnan(scale[1]).all()
    assert float(rstd[2]) == 0.0 and torch.isnan(h[2, 7]) and not h[2, 8:].any()
    assert torch.isnan(scale[2, 0]) and torch.all(scale[2, 1:] == 2.0 ** -126)
    assert abs(float(rstd[3]) * EPS ** 0.5 - 1) < 1e-6
    assert float(rstd[4]) == 0.0 and not h[4].any()
    ref, _ = on.forward(f64(x[5:]), np.ones(cols), EPS)
    _close("h", h[5:], ref, 70 * U * np.abs(ref))


# enough aligned rows for the staged form: one and several rows a block, two and four units a thread, one stage
STAGED = [(1000, 512, 0, 0), (777, 520, 8, 32), (610, 1024, 0, 0), (320, 4104, 24, 0), (310, 8192, 0, 0), (305, 12288, 0, 0),
          (308, 16384, 0, 0)]
# the same for rows that start off a unit, at every step between rows
STAGED_SHIFTED = [(2500, 515, 0, 0), (4000, 1013, 0, 0), (3333, 1030, 0, 0), (950, 4100, 0, 0), (1400, 2043, 3, 16),
                  (640, 6001, 0, 0), (620, 12285, 0, 0), (400, 16373, 0, 0)]


@pytest.mark.parametrize("rows,cols,pad,lead", SHAPES + SHIFTED + STAGED + STAGED_SHIFTED)
@pytest.mark.parametrize("at,st,gt,dgt,stream_grad,p", [
    (BF, BF, BF, F32, True, 0.0), (BF, F32, F32, BF, True, 0.1), (F32, F32, F32, F32, False, 0.25), (F32, BF, BF, F32, True, 0.0),
])
def test_add_rmsnorm_backward_matches_oracle(rows, cols, pad, lead, at, st, gt, dgt, stream_grad, p):
    dh, _ = _rows(rows, cols, pad, at, 21 + rows + cols, 1e-3, lead)
    s, _ = _rows(rows, cols, pad, st, 22 + rows + cols, 1.5, lead)
    ds, _ = _rows(rows, cols, pad, st, 23 + rows + cols, 1e-3, lead) if stream_grad else (None, None)
    gain = (1.0 + synth.normal((cols,), 0.2, 24 + cols)).to(gt).to(DEV)
    s64 = f64(s.float())
    rstd = torch.from_numpy((1.0 / np.sqrt((s64 ** 2).mean(axis=1) + EPS)).astype(np.float32)).to(DEV)
    dr, drb = _rows(rows, cols, pad, st, None, lead=lead)
    dx, dxb = _rows(rows, cols, pad, at, None, lead=lead)
    dg = torch.full((cols,), float("nan"), dtype=dgt, device=DEV)
    ws = torch.empty(native.sf_add_rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    args = dict(dsum=ds, dresidual=dr, dx=dx, dgain=dg, p=p, rng=native.rng(SEED, OFF), ws=ws)
    native.sf_add_rmsnorm_backward(dh, s, gain, rstd, **args)
    native.sf_sync_status()
    ref, rg, mag, gmag = on.backward(f64(dh.float()), s64, f64(gain.float()), EPS, None if ds is None else f64(ds.float()))
    _close("dresidual", dr, ref, _stored(st, ref, 96 * U * mag))
    kept = od.mask(rows, cols, p, SEED, OFF) if p else np.ones_like(ref, dtype=bool)
    f = od.factor(p) if p else 1.0
    rx = np.where(kept, ref * f, 0.0)
    _close("dx", dx, rx, np.where(kept, _stored(at, rx, 98 * U * mag * f), 0.0))
    _close("dgain", dg, rg, _stored(dgt, rg, 160 * U * gmag))
    assert _guard_ok(dr, drb, lead) and _guard_ok(dx, dxb, lead)
    # the same bits again, and dgain alone
    first = [t.clone() for t in (dr, dx, dg)]
    native.sf_add_rmsnorm_backward(dh, s, gain, rstd, **args)
    for a, b in zip(first, (dr, dx, dg)):
        assert torch.equal(a, b)
    dg.fill_(float("nan"))
    native.sf_add_rmsnorm_backward(dh, s, gain, rstd, dsum=ds, dgain=dg, ws=ws)
    assert torch.equal(dg, first[2])
    native.sf_sync_status()


def test_add_rmsnorm_backward_many_rows_and_no_rows():
    # more rows than resident blocks by far, so each block sums many rows of dgain
    rows, cols = 20000, 264
    dh, s = synth.normal((rows, cols), 1.0, 1).to(DEV), synth.normal((rows, cols), 1.0, 2).to(DEV)
    gain = torch.ones(cols, device=DEV)
    rstd = torch.rsqrt(s.double().square().mean(dim=1) + EPS).float()
    dg = torch.empty(cols, device=DEV)
    ws = torch.empty(native.sf_add_rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    native.sf_add_rmsnorm_backward(dh, s, gain, rstd, dgain=dg, ws=ws)
    _, rg, _, gmag = on.backward(f64(dh), f64(s), np.ones(cols), EPS)
    _close("dgain", dg, rg, 160 * U * gmag)
    e = torch.empty(0, cols, device=DEV)
    native.sf_add_rmsnorm_backward(e, e, gain, torch.empty(0, device=DEV), dresidual=e, dgain=dg, ws=ws)
    native.sf_sync_status()
    assert not dg.any()


@pytest.mark.parametrize("st", [BF, F32])
@pytest.mark.parametrize("rows,cols,pad", [(37, 1021, 2), (2500, 1021, 6), (700, 63, 4), (650, 4100, 1), (40, 16369, 4)])
def test_what_lies_beside_the_rows_stays_out(rows, cols, pad, st):
    # the same rows in a buffer whose padding is NaN
    def both(dtype, seed, std):
        v, _ = _rows(rows, cols, pad, dtype, seed, std)
        w = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device=DEV)[:, :cols]
        w.copy_(v)
        return v, w
    dh, s, ds = both(BF, 71, 1e-3), both(st, 72, 1.5), both(st, 73, 1e-3)
    gain = (1.0 + synth.normal((cols,), 0.2, 74)).to(DEV)
    rstd = torch.rsqrt(s[0].float().square().mean(dim=1) + EPS)
    ws = torch.empty(native.sf_add_rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    outs = []
    for i in range(2):
        dr, dx = _rows(rows, cols, pad, st)[0], _rows(rows, cols, pad, BF)[0]
        dg = torch.empty(cols, device=DEV)
        native.sf_add_rmsnorm_backward(dh[i], s[i], gain, rstd, dsum=ds[i], dresidual=dr, dx=dx, dgain=dg, p=0.1,
                                       rng=native.rng(SEED, OFF), ws=ws)
        outs.append((dr, dx, dg))
    native.sf_sync_status()
    for a, b in zip(*outs):
        assert torch.equal(a, b) and bool(torch.isfinite(a).all())


@pytest.mark.parametrize("rows,cols", [(130, 520), (400, 517), (2500, 1021)])
def test_sum_and_outputs_in_place(rows, cols):
    x, r = synth.normal((rows, cols), 1.0, 5, dtype=BF).to(DEV), synth.normal((rows, cols), 1.0, 6, dtype=BF).to(DEV)
    gain = torch.ones(cols, dtype=BF, device=DEV)
    s, h = torch.empty_like(r), torch.empty_like(x)
    native.sf_add_rmsnorm_forward(x, r, gain, EPS, sum=s, h=h)
    x2, r2 = x.clone(), r.clone()
    native.sf_add_rmsnorm_forward(x2, r2, gain, EPS, sum=r2, h=x2)
    assert torch.equal(r2, s) and torch.equal(x2, h)
    rstd = torch.rsqrt(s.float().square().mean(dim=1) + EPS)
    dr, dx = torch.empty_like(s), torch.empty_like(x)
    native.sf_add_rmsnorm_backward(h, s, gain, rstd, dsum=r, dresidual=dr, dx=dx)
    d1, d2 = h.clone(), r.clone()
    native.sf_add_rmsnorm_backward(d1, s, gain, rstd, dsum=d2, dresidual=d2, dx=d1)
    native.sf_sync_status()
    assert torch.equal(d1, dx) and torch.equal(d2, dr)


def test_on_another_stream():
    x = synth.normal((512, 1024), 1.0, 5, dtype=BF).to(DEV)
    gain = torch.ones(1024, device=DEV)
    want, got = torch.empty_like(x), torch.empty_like(x)
    native.sf_add_rmsnorm_forward(x, None, gain, EPS, h=want)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    native.sf_add_rmsnorm_forward(x, None, gain, EPS, h=got, stream=st)
    native.sf_sync_status(st)
    assert torch.equal(got, want)
