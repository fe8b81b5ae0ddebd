"""fp64 residual addition and root-mean-square norm (test infrastructure only).

s = r + x',  rstd = 1 / sqrt(mean(s^2) + eps),  h = s rstd g  (Zhang and
Sennrich 2019; SlideFormer lists a fused RMSNorm among its kernels and gives
no formula), its gradients, and the 8-bit form: per group of columns
scale = max(max |h| / 448, 2^-126), q = h / scale rounded to the nearest e4m3
value (4 exponent bits with bias 7, 3 fraction bits, subnormal quantum 2^-9,
largest value 448, ties to even).
"""

import numpy as np


def forward(s, gain, eps):
    s, gain = np.asarray(s, dtype=np.float64), np.asarray(gain, dtype=np.float64)
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    return s * rstd[:, None] * gain, rstd


def backward(dh, s, gain, eps, dsum=None):
    """ds, dgain and the magnitudes of their terms, rstd taken from s."""
    dh, s, gain = (np.asarray(v, dtype=np.float64) for v in (dh, s, gain))
    rstd = (1.0 / np.sqrt(np.mean(s * s, axis=1) + eps))[:, None]
    n = s * rstd
    dn = dh * gain
    ds = rstd * (dn - n * np.mean(dn * n, axis=1, keepdims=True))
    mag = rstd * (np.abs(dn) + np.abs(n) * np.mean(np.abs(dn * n), axis=1, keepdims=True))
    if dsum is not None:
        ds, mag = ds + dsum, mag + np.abs(dsum)
    return ds, (dh * n).sum(axis=0), mag, np.abs(dh * n).sum(axis=0)


def e4m3_quantum(v):
    """Distance between neighbouring e4m3 values around |v| <= 448."""
    _, e = np.frexp(np.asarray(v, dtype=np.float64))
    return np.ldexp(1.0, np.maximum(e - 4, -9))


def e4m3(v):
    q = e4m3_quantum(v)
    return np.clip(np.rint(np.asarray(v, dtype=np.float64) / q) * q, -448.0, 448.0)


def quantize(h, group):
    """(q, scale [rows, groups], scale per element) of h with one scale per `group` columns (0: per row)."""
    h = np.asarray(h, dtype=np.float64)
    rows, cols = h.shape
    width = group or cols
    n = -(-cols // width)
    scale = np.empty((rows, n))
    each = np.empty_like(h)
    for i in range(n):
        c = slice(i * width, min(cols, (i + 1) * width))
        scale[:, i] = np.maximum(np.abs(h[:, c]).max(axis=1) / 448.0, 2.0 ** -126)
        each[:, c] = scale[:, i:i + 1]
    return e4m3(h / each), scale, each
