"""Every form of a residual block's end and its checkpoints with what a call may bring to any of them (GPU): fp32 scales, one
operand as a checkpoint and the other in full, entries that are not finite.

Tolerances as in test_gpu_checkpoint.py and test_gpu_sandwich.py.  With fp32 scales value * scale is rounded once more, u =
2^-24: a fifth rounding of a loaded value; a gradient holds x and s at most eight times in all, 8u, less than a tenth of the
96u that the least of its bounds has.
"""

import numpy as np
import pytest
import torch

from _block_end import BF, DEV, E4, F32, U, close, guard_ok, make_checkpoint, new_checkpoint, rows_of, stored
from _util import f64
from layer_optimizer_gb300 import native, synth
from oracle import checkpoint as oc
from oracle import sandwich as osw
from test_gpu_sandwich import EPS, _check_backward, _gain, _gate, _np, _outputs

pytestmark = pytest.mark.gpu


def _fp32_checkpoint(rows, cols, group, seed, std=1.0, pad=0, lead=0):
    """(checkpoint, its values in fp64) of e4m3 codes and fp32 scales that are no powers of two."""
    q, _ = rows_of(rows, cols, pad, E4, None, lead=lead)
    q.copy_(synth.normal((rows, cols), 60.0, seed).clamp(-448, 448).to(E4))
    scale = ((synth.normal((rows, -(-cols // group) if group else 1), 0.2, seed + 1).abs() + 0.5) * (std / 60.0)).to(DEV)
    return native.checkpoint(q, scale, group), oc.restore(f64(q.float()), f64(scale), group)


LOADS = [(400, 1024, 0, 0), (3, 4096, 0, 0),              # whole units of 16 columns
         (64, 264, 8, 8), (300, 40, 0, 0),                # of eight
         (37, 1021, 0, 0), (64, 256, 3, 0), (33, 700, 0, 1),      # off them
         (300, 33, 7, 0), (7, 5, 0, 0)]                   # short


@pytest.mark.parametrize("rows,cols,pad,lead", LOADS)
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("yt,factors", [(BF, True), (F32, False)])
def test_load_with_fp32_scales(rows, cols, pad, lead, group, yt, factors):
    ck, ref = _fp32_checkpoint(rows, cols, group, 3 + cols, 1.0, pad, lead)
    y, buf = rows_of(rows, cols, pad, yt, None, lead=lead)
    f = torch.rand(rows, device=DEV) + 0.5 if factors else None
    gain = _gain(cols, BF, 5) if factors else None
    native.sf_checkpoint_load(ck, y, row_factor=f, gain=gain)
    native.sf_sync_status()
    if factors:
        ref = ref * f64(f)[:, None] * f64(gain.float())
    close("y", y, ref, stored(yt, ref, 5 * U * np.abs(ref)))
    assert guard_ok(y, buf, lead)


# few rows (of one step a thread, of two, of blocks of over 256 threads), many; on units, off them
BACK = [(5, 264), (5, 1003), (70, 4104), (9, 9000), (400, 1024), (400, 1032), (400, 1003), (333, 250), (1000, 72), (310, 8192), (310, 8200)]


def _back(rows, cols, st, gates, post, make_x, make_s, **without):
    """One backward call with x and s as make_* give them: (what the call has, their values in fp64)."""
    (xs, rx), (ss, rs) = make_x(), make_s()
    dh, ds = rows_of(rows, cols, 0, BF, 23 + cols, 1.0)[0], rows_of(rows, cols, 0, st, 24 + cols, 1.0)[0]
    g1, g2 = (_gain(cols, F32, 25) if post else None), _gain(cols, F32, 26)
    gate, span = _gate(rows, cols, gates, BF, 27)
    rho1 = torch.from_numpy(osw.rstd(rx, EPS)).float().to(DEV) if post else None
    rho2 = torch.from_numpy(osw.rstd(rs, EPS)).float().to(DEV)
    kw = dict(dh=dh, dsum=ds, x=xs, sum=ss, gain_post=g1, gain_pre=g2, gate=gate, rstd_post=rho1, rstd_pre=rho2)
    ref = osw.backward(_np(dh), _np(ds), rx, rs, _np(g1), _np(g2), _np(gate), span, 0.8, 0.5, _np(rho1), _np(rho2))
    out = _outputs(rows, cols, 0, 0, BF, st, kw)
    native.sf_sandwich_norm_backward(native.sandwich(EPS, 0.8, 0.5, 0.0, span), **kw, **out)
    native.sf_sync_status()
    _check_backward(out, {k: (g, 1.1 * mag) for k, (g, mag) in ref.items()}, BF, st)


@pytest.mark.parametrize("rows,cols", BACK)
@pytest.mark.parametrize("group,gates,post,st", [(0, 3, True, F32), (32, 10 ** 9, True, BF), (32, 0, False, BF), (128, 3, True, BF)])
def test_backward_with_fp32_scales(rows, cols, group, gates, post, st):
    _back(rows, cols, st, gates, post, lambda: _fp32_checkpoint(rows, cols, group, 31), lambda: _fp32_checkpoint(rows, cols, group, 33, 2.0))


@pytest.mark.parametrize("rows,cols", BACK)
@pytest.mark.parametrize("kept", ["x", "sum", "groups"])
@pytest.mark.parametrize("gates,post,st", [(3, True, F32), (10 ** 9, False, BF)])
def test_backward_with_operands_of_two_kinds(rows, cols, kept, gates, post, st):
    # a checkpoint of one, the other in full; or both, with scales of different kinds and groups
    def full(dtype, seed, std):
        t, _ = rows_of(rows, cols, 0, dtype, seed, std)
        return t, _np(t)

    def in8(seed, std):
        ck, q, scale = make_checkpoint(rows_of(rows, cols, 0, F32, seed, std)[0], 64)
        return ck, oc.restore(_np(q), _np(scale).reshape(rows, -1), 64)

    makes = {"x": (lambda: in8(41, 1.5), lambda: full(st, 42, 2.0)), "sum": (lambda: full(BF, 43, 1.5), lambda: in8(44, 2.0)),
             "groups": (lambda: in8(45, 1.5), lambda: _fp32_checkpoint(rows, cols, 0, 46, 2.0))}
    _back(rows, cols, st, gates, post, *makes[kept])


@pytest.mark.parametrize("rows,cols", [(400, 1024), (400, 1032), (400, 1003), (330, 2064), (310, 12288), (310, 12291), (20, 264), (300, 512)])
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("at,st", [(BF, BF), (F32, F32)])
def test_entries_that_are_not_finite(rows, cols, group, at, st):
    """In several rows of a block: checkpoints as defined, s as added, and every other row's bits as without them."""
    x0, r = rows_of(rows, cols, 0, at, 51, 1.0)[0], rows_of(rows, cols, 0, st, 52, 2.0)[0]
    x = x0.clone()
    top = torch.finfo(at).max
    x[1, 5], x[2, 7], x[3, cols - 1], x[4] = float("nan"), float("inf"), float("-inf"), float("inf")
    x[6, 33], x[6, 34], x[7, 200], x[8, :40], x[9] = float("nan"), float("inf"), top, float("-inf"), float("nan")
    x[rows - 1, 64], x[rows - 2, 3] = float("inf"), float("nan")
    if st == F32:
        r[5, 9] = float("inf")      # s alone
    else:
        r[7, 200] = top             # their sum is past fp32's largest, or next to it
    dirty = [1, 2, 3, 4, 5, 6, 7, 8, 9, rows - 2, rows - 1]
    clean = torch.ones(rows, dtype=torch.bool, device=DEV)
    clean[dirty] = False
    g = _gain(cols, F32, 53)

    def run(x):
        x8, q1, c1, _ = new_checkpoint(rows, cols, group)
        s8, q2, c2, _ = new_checkpoint(rows, cols, group)
        s, h = torch.empty(rows, cols, dtype=st, device=DEV), torch.empty(rows, cols, dtype=at, device=DEV)
        rho = torch.empty(rows, device=DEV)
        native.sf_sandwich_norm_forward(native.sandwich(EPS), x, r, gain_pre=g, sum=s, h=h, x8=x8, sum8=s8, rstd_pre=rho)
        native.sf_sync_status()
        return q1, c1, q2, c2, s, h, rho

    got, was = run(x), run(x0)
    for a, b in zip(got, was):
        bits = torch.int32 if a.element_size() == 4 else torch.int16 if a.element_size() == 2 else torch.uint8
        assert torch.equal(a.view(bits)[clean], b.view(bits)[clean])
    total = x.float() + r.float()      # one rounding, as r + x here
    for (q, c), v in (((got[0], got[1]), x.float()), ((got[2], got[3]), total)):
        rq, rs = oc.quantize(f64(v), group)
        assert np.array_equal(f64(c.float()).reshape(rs.shape), rs)
        assert np.array_equal(f64(q.float()), rq, equal_nan=True)
    assert np.array_equal(f64(got[4].float()), f64(total.to(st).float()), equal_nan=True)
    # with a norm after the block and one scale a row, the same checkpoint of x again
    x8, q, c, _ = new_checkpoint(rows, cols, group)
    h = torch.empty(rows, cols, dtype=at, device=DEV)
    native.sf_sandwich_norm_forward(native.sandwich(EPS), x, r, gain_post=g, gain_pre=g, h=h, x8=x8)
    native.sf_sync_status()
    assert torch.equal(q.view(torch.uint8), got[0].view(torch.uint8)) and torch.equal(c.view(torch.uint8), got[1].view(torch.uint8))
    assert bool(torch.isfinite(h[clean]).all())


# converted on the way, restored first (over several waves of tiles too), on the CUDA cores
@pytest.mark.parametrize("tokens,out,cin", [(130, 264, 256), (300, 1000, 1040), (520, 2048, 272), (700, 4400, 4352), (130, 264, 250)])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_weight_gradient_with_fp32_scales(tokens, out, cin, group):
    # X is value * scale rounded to fp32 and then to bf16; what follows is exact products and sums as of power-of-two scales
    ck, _ = _fp32_checkpoint(tokens, cin, group, 61)
    q, scale = ck.tensors
    n = group or cin
    x = (q.float() * scale.repeat_interleave(n, dim=1)[:, :cin]).to(BF).double()
    dy = synth.normal((tokens, out), 1.0, 62).to(BF).to(DEV)
    dw = torch.empty(out, cin, device=DEV)
    ws = torch.empty(max(16, native.sf_checkpoint_wgrad_workspace_bytes(tokens, out, cin)), dtype=torch.uint8, device=DEV)
    native.sf_checkpoint_wgrad(dy, ck, dw, ws=ws)
    native.sf_sync_status()
    ref, mag = dy.double().t() @ x, dy.double().abs().t() @ x.abs()
    assert bool(((dw.double() - ref).abs() <= 1e-5 * mag + U * ref.abs()).all())
