"""fp64 8-bit checkpoints (test infrastructure only).

Per group of columns (0: the row) the scale is 2^k, k the smallest integer >= -126
with max |v| <= 448 2^k over the finite entries, and an entry is v / 2^k rounded to
the nearest e4m3 value, ties to even; what is not finite is NaN.
"""

import numpy as np

from . import norm


def scales(v, group):
    """2^k per row and group."""
    v = np.asarray(v, dtype=np.float64)
    top = np.where(np.isfinite(v), np.abs(v), 0.0)
    width = group or v.shape[1]
    out = np.empty((v.shape[0], -(-v.shape[1] // width)))
    for i in range(out.shape[1]):
        m = top[:, i * width:(i + 1) * width].max(axis=1)
        k = np.full(m.shape, -126)
        while (m > np.ldexp(448.0, k)).any():
            k = k + (m > np.ldexp(448.0, k))
        out[:, i] = np.ldexp(1.0, k)
    return out


def spread(scale, group, cols):
    """Per element: its group's scale."""
    return np.repeat(np.asarray(scale, dtype=np.float64), group or cols, axis=1)[:, :cols]


def quantize(v, group):
    """(values, scales [rows, groups])."""
    v = np.asarray(v, dtype=np.float64)
    s = scales(v, group)
    fine = np.isfinite(v)
    q = norm.e4m3(np.where(fine, v, 0.0) / spread(s, group, v.shape[1]))
    return np.where(fine, q, np.nan), s


def restore(q, scale, group):
    q = np.asarray(q, dtype=np.float64)
    return q * spread(scale, group, q.shape[1])


def weight_grad(dy, x, base=None):
    """dW = base + dY^T X and the magnitudes of its terms."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    dw, mag = dy.T @ x, np.abs(dy).T @ np.abs(x)
    return (dw, mag) if base is None else (dw + base, mag + np.abs(base))
