"""The end of a residual block and its gradients against the fp64 oracle (GPU).

Tolerances, derived from the arithmetic (u = 2^-24, one fp32 rounding):

* rho1: a sum of positive squares, at most 4 x 9 additions a thread, 5 of lanes and 16 of warps, half of whose error
  passes to rho, a rounded mean, rsqrt within 2 ulp: 64u.
* s: rho1's error and five products of the branch (72u of it), two roundings of the sum.
* rho2: 64u and s's error through the squares.      h: rho2's error, two products, s's error.
* e4m3 outputs: half a quantum of the value under the kernel's own scale, and s's error; the scale is a power of two
  and the smallest that holds the group's maximum, up to s's error.
* d: a sum of up to 16384 signed terms in chains of 2 x 8, 5 and 32, and about ten more roundings: 96u of the terms'
  magnitudes.  dx: the same again through w: 192u.
* sums over rows: each chain adds at most the rows that one worker has and the partial rows / 32 + 37; the cases here
  stay below 64 + 128: 192u of the terms' magnitudes and d's 96u (d is a factor of dgain_post and dgate).
"""

import numpy as np
import pytest
import torch

from _block_end import BF, DEV, F32, SHAPES, U, close, guard_ok, make_checkpoint, new_checkpoint, rows_of, stored
from _util import f64
from layer_optimizer_gb300 import native, synth
from oracle import checkpoint as oc
from oracle import norm as on
from oracle import sandwich as osw

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _np(t):
    return None if t is None else f64(t.float())


def _gate(rows, cols, gates, dtype, seed, pad=0):
    """(gate, span) of `gates` rows (0: none), rows off their units with pad."""
    if not gates:
        return None, 0
    span = -(-rows // min(gates, rows))
    g, _ = rows_of(-(-rows // span), cols, pad, dtype)
    g.copy_((0.5 + synth.normal(tuple(g.shape), 0.3, seed)).to(dtype))
    return g, span


def _gain(cols, dtype, seed, offset=0.0):
    return (1.0 - offset + synth.normal((cols,), 0.2, seed)).to(dtype).to(DEV)


def _check_8(name, q, scale, ref, err, group):
    cols = ref.shape[1]
    k = f64(scale.float()).reshape(ref.shape[0], -1)
    assert np.array_equal(np.exp2(np.round(np.log2(k))), k)
    width = group or cols
    for i in range(k.shape[1]):
        c = slice(i * width, min(cols, (i + 1) * width))
        low = (np.abs(ref) - err)[:, c].max(axis=1)
        high = (np.abs(ref) + err)[:, c].max(axis=1)
        assert np.all(low <= 448 * k[:, i]) and np.all((high > 224 * k[:, i]) | (k[:, i] == 2.0 ** -126)), name
    each = oc.spread(k, group, cols)
    v = f64(q.float())
    quantum = on.e4m3_quantum(np.minimum(448.0, np.maximum(np.abs(v), np.abs(ref / each))))
    assert np.all(np.abs(v - ref / each) <= 0.5 * quantum + err / each), name


FORWARD = [
    # x and h, stream, vectors, gate rows, post, pre, residual, a, b, gain offset, group of the checkpoints
    (BF, BF, BF, 1, True, True, True, 1.0, 1.0, 0.0, 128),
    (BF, F32, F32, 4, True, True, True, 0.8, 0.25, 1.0, 32),
    (F32, BF, BF, 0, True, True, True, 1.0, 0.5, 0.0, 0),
    (F32, F32, F32, 10 ** 9, True, True, False, 1.0, 2.0, 1.0, 64),
    (BF, BF, F32, 3, False, True, True, -1.5, 1.0, 0.0, None),
    (BF, BF, BF, 0, True, False, True, 1.0, 1.0, 0.0, 32),
]


@pytest.mark.parametrize("rows,cols,pad,lead", SHAPES)
@pytest.mark.parametrize("at,st,gt,gates,post,pre,res,a,b,off,group", FORWARD)
def test_forward_matches_oracle(rows, cols, pad, lead, at, st, gt, gates, post, pre, res, a, b, off, group):
    x, _ = rows_of(rows, cols, pad, at, 11 + rows + cols, 1.5, lead)
    r, _ = rows_of(rows, cols, pad, st, 12 + rows + cols, 2.0, lead) if res else (None, None)
    g1, g2 = (_gain(cols, gt, 13, off) if post else None), (_gain(cols, gt, 14, off) if pre else None)
    gate, span = _gate(rows, cols, gates, gt, 15, pad)
    s, sbuf = rows_of(rows, cols, pad, st if res else at, None, lead=lead)
    h, hbuf = rows_of(rows, cols, pad, at, None, lead=lead) if pre else (None, None)
    x8 = s8 = None
    if group is not None:
        x8, q1, c1, b1 = new_checkpoint(rows, cols, group, pad, lead)
        s8, q2, c2, b2 = new_checkpoint(rows, cols, group, pad, lead)
    rho1 = torch.full((rows,), float("nan"), device=DEV) if post else None
    rho2 = torch.full((rows,), float("nan"), device=DEV) if pre else None
    native.sf_sandwich_norm_forward(native.sandwich(EPS, a, b, off, span), x, r, gain_post=g1, gain_pre=g2, gate=gate, sum=s, h=h,
                                    x8=x8, sum8=s8, rstd_post=rho1, rstd_pre=rho2)
    native.sf_sync_status()
    plus = lambda g: None if g is None else _np(g) + off  # noqa: E731
    f = osw.forward(_np(x), _np(r), plus(g1), plus(g2), _np(gate), span, a, b, EPS)
    es = 72 * U * np.abs(f["branch"]) + 2 * U * (np.abs(f["s"]) + np.abs(f["branch"]))
    close("sum", s, f["s"], stored(s.dtype, f["s"], es))
    assert guard_ok(s, sbuf, lead)
    if post:
        close("rstd_post", rho1, f["rho1"], 64 * U * f["rho1"])
    if pre:
        rel = 64 * U + np.mean(es * np.abs(f["s"]), axis=1) * f["rho2"] ** 2
        close("rstd_pre", rho2, f["rho2"], rel * f["rho2"])
        eh = np.abs(f["h"]) * (rel + 4 * U)[:, None] + es * f["rho2"][:, None] * np.abs(plus(g2))
        close("h", h, f["h"], stored(at, f["h"], eh))
        assert guard_ok(h, hbuf, lead)
    if group is not None:
        rq, rs = oc.quantize(_np(x), group)
        assert np.array_equal(f64(q1.float()), rq) and np.array_equal(f64(c1.float()).reshape(rs.shape), rs)
        _check_8("sum8", q2, c2, f["s"], es, group)
        assert guard_ok(q1, b1, lead) and guard_ok(q2, b2, lead)


BACKWARD = [
    # act, stream, vectors, gate rows, post, dh, dsum, group of the checkpoints (None: full), a, b, gain offset
    (BF, BF, BF, 1, True, True, True, None, 1.0, 1.0, 0.0),
    (BF, F32, F32, 4, True, True, True, 128, 0.8, 0.25, 1.0),
    (F32, F32, F32, 0, True, True, False, None, 1.0, 1.0, 0.0),
    (BF, BF, BF, 10 ** 9, True, True, True, 32, 1.0, 0.5, 0.0),
    (F32, BF, BF, 3, False, True, True, 0, -1.5, 2.0, 1.0),
    (BF, BF, F32, 2, True, False, True, None, 1.0, 1.0, 0.0),
]


def _backward_case(rows, cols, pad, lead, at, st, gt, gates, post, pre, has_dsum, group, a, b, off, seed=0):
    x, _ = rows_of(rows, cols, pad, at, 21 + rows + cols + seed, 1.5, lead)
    s, _ = rows_of(rows, cols, pad, st, 22 + rows + cols + seed, 2.0, lead)
    dh = rows_of(rows, cols, pad, at, 23 + rows + cols + seed, 1.0, lead)[0] if pre else None
    ds = rows_of(rows, cols, pad, st, 24 + rows + cols + seed, 1.0, lead)[0] if has_dsum else None
    g1, g2 = (_gain(cols, gt, 25, off) if post else None), (_gain(cols, gt, 26, off) if pre else None)
    gate, span = _gate(rows, cols, gates, gt, 27, pad)
    rho1 = torch.rsqrt(x.double().square().mean(1) + EPS).float() if post else None
    rho2 = torch.rsqrt(s.double().square().mean(1) + EPS).float() if pre else None
    xs, ss = x, s
    if group is not None:
        xs, q, c = make_checkpoint(x, group, pad, lead)
        rx = oc.restore(_np(q), _np(c).reshape(rows, -1), group)
        ss, q, c = make_checkpoint(s, group, pad, lead)
        rs = oc.restore(_np(q), _np(c).reshape(rows, -1), group)
    else:
        rx, rs = _np(x), _np(s)
    plus = lambda g: None if g is None else _np(g) + off  # noqa: E731
    ref = osw.backward(_np(dh), _np(ds), rx, rs, plus(g1), plus(g2), _np(gate), span, a, b, _np(rho1), _np(rho2))
    kw = dict(dh=dh, dsum=ds, x=xs, sum=ss if pre else None, gain_post=g1, gain_pre=g2, gate=gate, rstd_post=rho1, rstd_pre=rho2)
    return native.sandwich(EPS, a, b, off, span), kw, ref


def _outputs(rows, cols, pad, lead, at, st, kw, vt=F32):
    out = dict(dresidual=rows_of(rows, cols, pad, st, None, lead=lead)[0], dx=rows_of(rows, cols, pad, at, None, lead=lead)[0])
    if kw["dh"] is not None:
        out["dgain_pre"] = torch.full((cols,), float("nan"), dtype=vt, device=DEV)
    if kw["gain_post"] is not None:
        out["dgain_post"] = torch.full((cols,), float("nan"), dtype=vt, device=DEV)
    if kw["gate"] is not None:
        out["dgate"] = rows_of(kw["gate"].shape[0], cols, pad, vt)[0]
    out["ws"] = torch.full((native.sf_sandwich_norm_workspace_bytes(rows, cols),), 255, dtype=torch.uint8, device=DEV)
    return out


def _check_backward(out, ref, at, st, vt=F32):
    names = dict(dresidual=("dr", st, 96), dx=("dx", at, 192), dgain_pre=("dg2", vt, 192), dgain_post=("dg1", vt, 288),
                 dgate=("dgate", vt, 288))
    for k, (r, dtype, n) in names.items():
        if out.get(k) is not None:
            g, mag = ref[r]
            close(k, out[k], g, stored(dtype, g, n * U * mag))


@pytest.mark.parametrize("rows,cols,pad,lead", SHAPES)
@pytest.mark.parametrize("at,st,gt,gates,post,pre,has_dsum,group,a,b,off", BACKWARD)
def test_backward_matches_oracle(rows, cols, pad, lead, at, st, gt, gates, post, pre, has_dsum, group, a, b, off):
    p, kw, ref = _backward_case(rows, cols, pad, lead, at, st, gt, gates, post, pre, has_dsum, group, a, b, off)
    out = _outputs(rows, cols, pad, lead, at, st, kw)
    native.sf_sandwich_norm_backward(p, **kw, **out)
    native.sf_sync_status()
    _check_backward(out, ref, at, st)


# gate rows against workers: one each, several parts, more than there are workers, ragged last ones
@pytest.mark.parametrize("rows,cols,gates", [(1999, 256, 1), (1999, 256, 2), (1999, 256, 31), (1999, 256, 33), (5000, 1024, 777),
                                             (3001, 2048, 3001), (3001, 2051, 1501), (2500, 4096, 601), (1300, 9000, 160), (1300, 16384, 153)])
@pytest.mark.parametrize("post", [True, False])
def test_gate_rows_of_every_length(rows, cols, gates, post):
    p, kw, ref = _backward_case(rows, cols, 0, 0, BF, BF, F32, gates, post, True, True, None, 1.0, 0.5, 0.0)
    out = _outputs(rows, cols, 0, 0, BF, BF, kw)
    native.sf_sandwich_norm_backward(p, **kw, **out)
    native.sf_sync_status()
    _check_backward(out, ref, BF, BF)
    f = {k: v.clone() for k, v in out.items()}
    native.sf_sandwich_norm_backward(p, **kw, **out)
    assert all(torch.equal(f[k], out[k]) for k in f if k != "ws")          # the same bits again


@pytest.mark.parametrize("want", ["dresidual", "dx", "dgain_post", "dgain_pre", "dgate"])
@pytest.mark.parametrize("rows,cols", [(70, 264), (400, 1003)])
def test_single_gradients_in_bf16(want, rows, cols):
    p, kw, ref = _backward_case(rows, cols, 0, 0, BF, BF, BF, 3, True, True, True, None, 1.0, 0.5, 0.0)
    out = _outputs(rows, cols, 0, 0, BF, BF, kw, BF)
    native.sf_sandwich_norm_backward(p, **kw, **{k: v for k, v in out.items() if k in (want, "ws")})
    native.sf_sync_status()
    _check_backward({want: out[want]}, ref, BF, BF, BF)


@pytest.mark.parametrize("rows,cols,pad", [(3, 264, 0), (5, 1003, 3), (500, 1024, 0), (400, 1003, 1), (330, 8192, 8), (310, 12288, 0), (700, 72, 0)])
@pytest.mark.parametrize("group", [None, 0, 64])
def test_outputs_over_their_inputs(rows, cols, pad, group):
    """s over the residual and h over x, or s over x and h over the residual, or s over a gate row for each row: the bits of
    separate outputs."""
    x, r, gate = (rows_of(rows, cols, pad, BF, seed)[0] for seed in (31, 32, 33))
    g = torch.ones(cols, device=DEV)

    def run(x, r, gate, s, h):
        made = [new_checkpoint(rows, cols, group, 0, 0) for _ in range(2)] if group is not None else [(None,) * 4] * 2
        native.sf_sandwich_norm_forward(native.sandwich(EPS, gate_span=1), x, r, gain_post=g, gain_pre=g, gate=gate, sum=s, h=h,
                                        x8=made[0][0], sum8=made[1][0])
        native.sf_sync_status()
        return [s, h] + [m[i].view(torch.uint8) for m in made for i in (1, 2) if m[i] is not None]

    def again(t):      # with the same stride
        c = rows_of(rows, cols, pad, BF, None)[0]
        c.copy_(t)
        return c

    want = run(x, r, gate, rows_of(rows, cols, pad, BF, None)[0], rows_of(rows, cols, pad, BF, None)[0])
    assert bool(torch.isfinite(want[0].float()).all()) and bool(torch.isfinite(want[1].float()).all())
    for sum_over, h_over in (("r", "x"), ("x", "r"), ("gate", "x")):
        into = {"x": again(x), "r": again(r), "gate": again(gate)}
        got = run(into["x"], into["r"], into["gate"], into[sum_over], into[h_over])
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (sum_over, h_over)


def test_gradients_over_their_inputs():
    rows, cols = 500, 1024
    p, kw, ref = _backward_case(rows, cols, 0, 0, BF, BF, BF, 2, True, True, True, None, 1.0, 0.5, 0.0)
    out = _outputs(rows, cols, 0, 0, BF, BF, kw)
    out["dresidual"], out["dx"] = kw["dsum"], kw["dh"]
    native.sf_sandwich_norm_backward(p, **kw, **out)
    _check_backward(out, ref, BF, BF)
    p, kw, ref = _backward_case(rows, cols, 0, 0, BF, BF, BF, 2, True, True, True, None, 1.0, 0.5, 0.0)
    out["dresidual"], out["dx"] = kw["sum"], kw["x"]
    native.sf_sandwich_norm_backward(p, **kw, **out)
    _check_backward(out, ref, BF, BF)


@pytest.mark.parametrize("rows,cols,gates", [(500, 1024, 2), (700, 1024, 650), (64, 264, 3), (900, 72, 900), (400, 1003, 2), (3000, 264, 1500)])
def test_the_gates_gradient_over_the_gate(rows, cols, gates):
    p, kw, ref = _backward_case(rows, cols, 0, 0, BF, BF, F32, gates, True, True, True, None, 1.0, 0.5, 0.0)
    out = _outputs(rows, cols, 0, 0, BF, BF, kw)
    out["dgate"] = kw["gate"]
    native.sf_sandwich_norm_backward(p, **kw, **out)
    native.sf_sync_status()
    _check_backward(out, ref, BF, BF)


def test_two_streams_at_once():
    made = []
    for rows, cols, gates, group in ((2000, 2048, 3, 64), (777, 1003, 0, None)):
        p, kw, ref = _backward_case(rows, cols, 0, 0, BF, BF, BF, gates, True, True, True, group, 1.0, 0.5, 0.0)
        made.append((p, kw, ref, _outputs(rows, cols, 0, 0, BF, BF, kw), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for p, kw, ref, out, stream in made:
            native.sf_sandwich_norm_backward(p, **kw, **out, stream=stream)
    torch.cuda.synchronize()
    for p, kw, ref, out, stream in made:
        _check_backward(out, ref, BF, BF)


def test_pinned_host_rows_give_the_formulas_results():
    rows, cols = 400, 1024
    p, kw, ref = _backward_case(rows, cols, 0, 0, BF, BF, F32, 2, True, True, True, None, 1.0, 0.5, 0.0)
    out = _outputs(rows, cols, 0, 0, BF, BF, kw)
    for k in ("dh", "dsum", "x", "sum"):
        kw[k] = kw[k].cpu().contiguous().pin_memory()
    for k in ("dresidual", "dx"):
        out[k] = torch.empty(rows, cols, dtype=BF).pin_memory()
    native.sf_sandwich_norm_backward(p, **kw, **out)
    native.sf_sync_status()
    _check_backward(out, ref, BF, BF)
    x, r, h, s = kw["x"], kw["sum"], out["dx"], out["dresidual"]
    g = torch.ones(cols, device=DEV)
    native.sf_sandwich_norm_forward(native.sandwich(EPS), x, r, gain_post=g, gain_pre=g, sum=s, h=h)
    native.sf_sync_status()
    f = osw.forward(_np(x), _np(r), np.ones(cols), np.ones(cols), None, 0, 1.0, 1.0, EPS)
    es = 72 * U * np.abs(f["branch"]) + 2 * U * (np.abs(f["s"]) + np.abs(f["branch"]))
    close("sum", s, f["s"], stored(BF, f["s"], es))


@pytest.mark.parametrize("rows,cols,pad", [(400, 1024, 8), (400, 2064, 8), (400, 1024, 4), (320, 5008, 1), (310, 8192, 8), (330, 257, 0), (5000, 256, 8)])
@pytest.mark.parametrize("group", [None, 0, 32, 128])
def test_rows_next_to_units(rows, cols, pad, group):
    # rows on units of 8 or 4 columns, off them, many enough for every form
    x, _ = rows_of(rows, cols, pad, BF, 61, 1.5)
    r, _ = rows_of(rows, cols, pad, F32, 62, 2.0)
    g = _gain(cols, BF, 63)
    gate, span = _gate(rows, cols, 3, BF, 64)
    s, sbuf = rows_of(rows, cols, pad, F32)
    h, hbuf = rows_of(rows, cols, pad, BF)
    x8 = s8 = None
    if group is not None:
        x8, q1, c1, b1 = new_checkpoint(rows, cols, group, pad)
        s8, q2, c2, b2 = new_checkpoint(rows, cols, group, pad)
    rho1, rho2 = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    p = native.sandwich(EPS, 1.0, 0.5, 0.0, span)
    native.sf_sandwich_norm_forward(p, x, r, gain_post=g, gain_pre=g, gate=gate, sum=s, h=h, x8=x8, sum8=s8, rstd_post=rho1, rstd_pre=rho2)
    native.sf_sync_status()
    f = osw.forward(_np(x), _np(r), _np(g), _np(g), _np(gate), span, 1.0, 0.5, EPS)
    es = 72 * U * np.abs(f["branch"]) + 2 * U * (np.abs(f["s"]) + np.abs(f["branch"]))
    close("sum", s, f["s"], stored(F32, f["s"], es))
    rel = 64 * U + np.mean(es * np.abs(f["s"]), axis=1) * f["rho2"] ** 2
    close("h", h, f["h"], stored(BF, f["h"], np.abs(f["h"]) * (rel + 4 * U)[:, None] + es * f["rho2"][:, None] * np.abs(_np(g))))
    assert guard_ok(s, sbuf) and guard_ok(h, hbuf)
    if group is not None:
        rq, rs = oc.quantize(_np(x), group)
        assert np.array_equal(f64(q1.float()), rq) and np.array_equal(f64(c1.float()).reshape(rs.shape), rs)
        _check_8("sum8", q2, c2, f["s"], es, group)
        assert guard_ok(q1, b1) and guard_ok(q2, b2)
    p, kw, ref = _backward_case(rows, cols, pad, 0, BF, F32, BF, 3, True, True, True, group, 1.0, 0.5, 0.0)
    out = _outputs(rows, cols, pad, 0, BF, F32, kw)
    native.sf_sandwich_norm_backward(p, **kw, **out)
    native.sf_sync_status()
    _check_backward(out, ref, BF, F32)


def test_no_rows():
    cols = 72
    e = torch.empty(0, cols, dtype=BF, device=DEV)
    g = torch.ones(cols, dtype=BF, device=DEV)
    v = torch.empty(0, device=DEV)
    gate = torch.ones(1, cols, device=DEV)
    native.sf_sandwich_norm_forward(native.sandwich(EPS), e, e, gain_post=g, gain_pre=g, gate=gate, sum=e, h=e, rstd_pre=v)
    ws = torch.empty(native.sf_sandwich_norm_workspace_bytes(0, cols), dtype=torch.uint8, device=DEV)
    d1, d2, dg = torch.ones(cols, device=DEV), torch.ones(cols, device=DEV), torch.ones(1, cols, device=DEV)
    native.sf_sandwich_norm_backward(native.sandwich(EPS), dh=e, dsum=e, x=e, sum=e, gain_post=g, gain_pre=g, gate=gate, rstd_post=v,
                                     rstd_pre=v, dresidual=e, dx=e, dgain_post=d1, dgain_pre=d2, dgate=dg, ws=ws)
    native.sf_sync_status()
    assert not d1.any() and not d2.any() and not dg.any()


@pytest.mark.parametrize("cols", [256, 251])
def test_special_values_stay_in_their_rows(cols):
    rows = 9
    x = synth.normal((rows, cols), 1.0, 31).to(BF).to(DEV)
    r = synth.normal((rows, cols), 1.0, 32).to(BF).to(DEV)
    x[0], r[0] = 0.0, 0.0                           # nothing but zeros: rho = eps^-1/2
    x[1, 5], x[2, 7], x[3] = float("nan"), float("inf"), 3e38
    g = torch.ones(cols, device=DEV)
    s, h = torch.empty_like(x), torch.empty_like(x)
    rho1, rho2 = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ck, q, scale, _ = new_checkpoint(rows, cols, 32)
    native.sf_sandwich_norm_forward(native.sandwich(EPS), x, r, gain_post=g, gain_pre=g, sum=s, h=h, sum8=ck, rstd_post=rho1, rstd_pre=rho2)
    native.sf_sync_status()
    assert not h[0].any() and not s[0].any() and abs(rho1[0].item() - EPS ** -0.5) < 1e-4
    assert s[1].isnan().all() and h[1].isnan().all() and q[1].float().isnan().all()
    assert s[2].isnan().sum() == 1 and h[2].isnan().all()      # inf * 0; the others are r
    assert torch.equal(s[3], r[3])                             # squares past fp32's largest: rho1 0
    assert torch.isfinite(h[4:]).all() and torch.isfinite(s[4:]).all()
    f = osw.forward(_np(x[4:]), _np(r[4:]), np.ones(cols), np.ones(cols), None, 0, 1.0, 1.0, EPS)
    assert np.all(np.abs(_np(h[4:]) - f["h"]) <= 2.0 ** -8 * np.abs(f["h"]) + 1e-5)
    # the row with a NaN poisons the sums over rows, as in the formula, and no other row's gradients
    dh = synth.normal((rows, cols), 1.0, 33).to(BF).to(DEV)
    dx, dr = torch.empty_like(x), torch.empty_like(x)
    native.sf_sandwich_norm_backward(native.sandwich(EPS), dh=dh, x=x, sum=s, gain_post=g, gain_pre=g, rstd_post=rho1, rstd_pre=rho2,
                                     dresidual=dr, dx=dx)
    assert torch.isfinite(dx[4:]).all() and torch.isfinite(dr[4:]).all() and dx[1].isnan().all()


def test_backward_in_a_graph_and_on_a_side_stream():
    rows, cols = 300, 520
    p, kw, ref = _backward_case(rows, cols, 0, 0, BF, BF, BF, 5, True, True, True, 32, 1.0, 0.5, 0.0)
    out = _outputs(rows, cols, 0, 0, BF, BF, kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        native.sf_sandwich_norm_backward(p, **kw, **out)
    side.synchronize()
    _check_backward(out, ref, BF, BF)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        native.sf_sandwich_norm_backward(p, **kw, **out)
    for v in out.values():
        v.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    _check_backward(out, ref, BF, BF)


def test_past_2_31_elements():
    rows, cols = 270001, 8192
    x = torch.empty(rows, cols, dtype=BF, device=DEV)
    synth.fill_normal_(x, 1.0, 41)
    r = torch.empty_like(x)
    synth.fill_normal_(r, 1.0, 42)
    g = _gain(cols, F32, 43)
    gate = torch.rand(rows // 1000 + 1, cols, device=DEV) + 0.5
    s, h = torch.empty_like(x), torch.empty_like(x)
    rho1, rho2 = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    p = native.sandwich(EPS, 1.0, 0.5, 0.0, 1000)
    native.sf_sandwich_norm_forward(p, x, r, gain_post=g, gain_pre=g, gate=gate, sum=s, h=h, rstd_post=rho1, rstd_pre=rho2)
    native.sf_sync_status()
    pick = [0, 999, 1000, 262143, 262144, 262145, rows - 1]
    one = gate[[i // 1000 for i in pick]]
    f = osw.forward(_np(x[pick]), _np(r[pick]), _np(g), _np(g), _np(one), 1, 1.0, 0.5, EPS)
    es = 72 * U * np.abs(f["branch"]) + 2 * U * (np.abs(f["s"]) + np.abs(f["branch"]))
    close("sum", s[pick], f["s"], stored(BF, f["s"], es))
    dr, dx = r, torch.empty_like(x)
    ref = osw.backward(_np(h[pick]), None, _np(x[pick]), _np(s[pick]), _np(g), _np(g), _np(one), 1, 1.0, 0.5, _np(rho1[pick]), _np(rho2[pick]))
    native.sf_sandwich_norm_backward(p, dh=h, x=x, sum=s, gain_post=g, gain_pre=g, gate=gate, rstd_post=rho1, rstd_pre=rho2, dresidual=dr,
                                     dx=dx)
    native.sf_sync_status()
    _check_backward(dict(dresidual=dr[pick], dx=dx[pick]), ref, BF, BF)


@pytest.mark.parametrize("rows,cols,pad", [(9, 1024, 0), (9, 1003, 0), (400, 1024, 0), (400, 1032, 0), (400, 1003, 0), (310, 12288, 0)])
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("at", [BF, F32])
def test_checkpoints_keep_the_sign_of_zero(rows, cols, pad, group, at):
    x, r = (rows_of(rows, cols, pad, at, 71 + i, 1.0)[0] for i in range(2))
    for t in (x, r):      # s = r + x, -0 + -0 = -0
        t[:, 1::3] = -0.0
        t[:, 2::9] = 0.0
        t[:, 5::9] = -2.0 ** -30
        t[4::4, 7] = float("inf")
        t[5] = -0.0
    g = torch.ones(cols, device=DEV)
    x8, q1, _, _ = new_checkpoint(rows, cols, group)
    s8, q2, _, _ = new_checkpoint(rows, cols, group)
    h = torch.empty(rows, cols, dtype=at, device=DEV)
    native.sf_sandwich_norm_forward(native.sandwich(EPS), x, r, gain_pre=g, h=h, x8=x8, sum8=s8)
    native.sf_sync_status()
    for q, v in ((q1, x), (q2, x.float() + r.float())):
        fine = torch.isfinite(v)
        assert torch.equal((q.view(torch.uint8) >> 7)[fine].bool(), torch.signbit(v)[fine])
