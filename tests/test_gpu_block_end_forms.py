"""Every form of a residual block's end and its checkpoints with what a call may bring to any of them (GPU).
"""

import numpy as np
import pytest
import torch

from _block_end import BF, DEV, F32, new_checkpoint, rows_of
from _util import f64
from layer_optimizer_gb300 import native
from oracle import checkpoint as oc
from test_gpu_sandwich import EPS, _gain

pytestmark = pytest.mark.gpu


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
