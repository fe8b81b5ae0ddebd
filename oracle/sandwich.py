"""fp64 end of a residual block (test infrastructure only).

n = x rho1 g1 (or x),  s = a r + b gate n,  h = s rho2 g2,  rho = 1 / sqrt(mean(row^2) + eps);
row i takes row i // span of the gate.  The gradients are written term by term, with the
sum of the magnitudes of what is added beside each.
"""

import numpy as np


def _64(*vs):
    return [None if v is None else np.asarray(v, dtype=np.float64) for v in vs]


def rstd(x, eps):
    return 1.0 / np.sqrt(np.mean(x * x, axis=1) + eps)


def each_row(gate, span, rows):
    """The gate's row of every row (None: ones)."""
    if gate is None:
        return np.ones((rows, 1))
    return np.asarray(gate, dtype=np.float64)[np.arange(rows) // (span or max(1, rows))]


def forward(x, r, g1, g2, gate, span, a, b, eps):
    """{s, h, rho1, rho2, branch: b gate n}; h and the rhos None without their gains."""
    x, r, g1, g2 = _64(x, r, g1, g2)
    rho1 = None if g1 is None else rstd(x, eps)
    n = x if g1 is None else x * rho1[:, None] * g1
    branch = b * each_row(gate, span, len(x)) * n
    s = branch if r is None else a * r + branch
    rho2 = None if g2 is None else rstd(s, eps)
    h = None if g2 is None else s * rho2[:, None] * g2
    return dict(s=s, h=h, rho1=rho1, rho2=rho2, branch=branch)


def backward(dh, dsum, x, s, g1, g2, gate, span, a, b, rho1, rho2):
    """{name: (gradient, magnitude)}: dr, dx, dg1, dg2, dgate, with the given rhos."""
    dh, dsum, x, s, g1, g2, rho1, rho2 = _64(dh, dsum, x, s, g1, g2, rho1, rho2)
    rows, cols = (dh if dh is not None else dsum).shape
    d, mag, out = np.zeros((rows, cols)), np.zeros((rows, cols)), {}
    if dsum is not None:
        d, mag = d + dsum, mag + np.abs(dsum)
    if dh is not None:
        p = rho2[:, None]
        dn = dh * g2
        c = p ** 3 * np.mean(dn * s, axis=1, keepdims=True)
        c_mag = p ** 3 * np.mean(np.abs(dn * s), axis=1, keepdims=True)
        d, mag = d + p * dn - c * s, mag + p * np.abs(dn) + c_mag * np.abs(s)
        out["dg2"] = (dh * s * p).sum(axis=0), np.abs(dh * s * p).sum(axis=0)
    out["dr"] = a * d, abs(a) * mag
    gates = each_row(gate, span, rows)
    p = 1.0 if g1 is None else rho1[:, None]
    e, e_mag = b * d * gates, abs(b) * mag * np.abs(gates)
    if g1 is None:
        out["dx"] = e, e_mag
    else:
        w, w_mag = e * g1, e_mag * np.abs(g1)
        out["dx"] = (p * w - p ** 3 * x * np.mean(w * x, axis=1, keepdims=True),
                     p * w_mag + p ** 3 * np.abs(x) * np.mean(w_mag * np.abs(x), axis=1, keepdims=True))
        out["dg1"] = (e * x * p).sum(axis=0), (e_mag * np.abs(x) * p).sum(axis=0)
    if gate is not None and x is not None:
        n = x * p * (1.0 if g1 is None else g1)
        at = np.arange(rows) // (span or max(1, rows))
        total, t_mag = np.zeros(np.shape(gate)), np.zeros(np.shape(gate))
        np.add.at(total, at, b * d * n)
        np.add.at(t_mag, at, abs(b) * mag * np.abs(n))
        out["dgate"] = total, t_mag
    return out
