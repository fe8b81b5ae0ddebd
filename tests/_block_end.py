"""Inputs and comparisons shared by the tests of a residual block's end."""

import numpy as np
import torch

from _util import f64
from layer_optimizer_gb300 import native, synth

DEV = "cuda"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
E4, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
FILL = 7.0


def rows_of(rows, cols, pad, dtype, seed=None, std=1.0, lead=0):
    """A [rows, cols] view inside a wider, guarded buffer (lead extra elements in front, pad behind every row)."""
    buf = torch.full((lead + rows * (cols + pad) + 64,), FILL, dtype=F32, device=DEV).to(dtype)
    v = buf[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    if seed is not None:
        v.copy_(synth.normal((rows, cols), std, seed).to(dtype))
    return v, buf


def guard_ok(view, buf, lead=0):
    """Everything around the view still holds the fill."""
    rows, cols = view.shape
    b = buf.float().clone()
    b[lead:lead + rows * view.stride(0)].view(rows, -1)[:, :cols] = FILL
    return bool((b == FILL).all())


def stored(dtype, ref, err):
    """Bound of a value known within err and stored in dtype: err plus half a unit in its last place."""
    _, e = np.frexp(np.abs(ref) + err)
    least = -133 if dtype == BF else -149
    return err + np.ldexp(0.5, np.maximum(e - (8 if dtype == BF else 24), least))


def close(name, got, ref, bound):
    got = f64(got.float())
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(np.max(err / np.maximum(bound, 1e-300))), np.argwhere(bad)[:3])


def new_checkpoint(rows, cols, group, pad=0, lead=0):
    """(checkpoint, values, scales, buffer): scales start as NaN."""
    q, buf = rows_of(rows, cols, pad, E4, None, lead=lead)
    n = -(-cols // group) if group else 1
    scale = torch.full((rows, n), 255, dtype=torch.uint8, device=DEV).view(E8)
    return native.checkpoint(q, scale, group), q, scale, buf


def make_checkpoint(v, group, pad=0, lead=0):
    """A checkpoint of the tensor v through the library."""
    ck, q, scale, _ = new_checkpoint(v.shape[0], v.shape[1], group, pad, lead)
    native.sf_checkpoint_store(v, ck)
    return ck, q, scale


SHAPES = [
    (1, 1, 0, 0), (1, 7, 0, 0), (3, 8, 0, 0), (2, 4096, 0, 0), (1, 16384, 0, 0), (5, 1000, 0, 0),
    (37, 1021, 0, 0),        # odd rows: off their units from the second row on
    (300, 33, 7, 0),         # many short rows in a padded buffer
    (64, 256, 3, 0),         # a leading dimension off the unit
    (64, 256, 8, 1),         # a base off the unit
    (700, 128, 0, 0), (400, 2048, 16, 8), (161, 2056, 0, 0), (40, 16377, 0, 0), (900, 3, 0, 0), (333, 130, 6, 0),
    (620, 8192, 0, 0), (310, 12296, 0, 0),
]
