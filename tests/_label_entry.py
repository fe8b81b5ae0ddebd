"""Bounds of the cross-entropy's gradients that hold the label's entry p - 1 to its own size.

dZ = (p - onehot) / n is rounded to bf16 entry by entry, the last piece's
exponentials once more before that; the label's entry is p - 1 in fp32, rounded
once.  So an entry v of a row may be off by

  label's entry   |p - 1| (2^-8 + 1e-5) + p (2 z_err + 1e-5)
  any other       p (2 2^-8 + 2e-5 + 2 z_err)

(z_err = 1e-5 of sum |h||w|, the products' bound; 1e-5 the exponential's and the
log-sum-exp's), and dH and dW by those errors through |W| and |H|, 1e-5 of
|dZ||W| and |dZ|^T|H| for the sums, and half a unit in the last place where
stored in bf16.  Where the model is sure, p 2^-8 at the label would be far more
than the entry itself.
"""

import numpy as np

from oracle.lce import lce


def half_ulp(x, bf16):
    _, e = np.frexp(x)
    return np.ldexp(0.5, e - (8 if bf16 else 24))


def bounds(H, W, y, bf16=(False, False)):
    """{"dH": (reference, bound), "dW": ...} of fp64 H, W and labels (all tokens labelled, or -100)."""
    y = np.asarray(y)
    on = y >= 0
    res = lce(H, W, y)
    n = max(1, res["n"])
    rows = np.flatnonzero(on)
    z_err = 1e-5 * (np.abs(H) @ np.abs(W).T)
    P = np.exp(res["Z"] - res["lse"][:, None]) * on[:, None]
    eZ = P * (2 * 2.0 ** -8 + 2e-5 + 2 * z_err)
    p = P[rows, y[rows]]
    eZ[rows, y[rows]] = np.abs(np.expm1(res["Z"] - res["lse"][:, None])[rows, y[rows]]) * (2.0 ** -8 + 1e-5) \
        + p * (2 * z_err[rows, y[rows]] + 1e-5)
    eZ = eZ / n + 1e-5 * np.abs(res["dZ"])
    out = {}
    for name, err, b in (("dH", eZ @ np.abs(W), bf16[0]), ("dW", eZ.T @ np.abs(H), bf16[1])):
        out[name] = (res[name], err + half_ulp(np.abs(res[name]) + err, b) + 1e-38)
    return out


def outside(H, W, y, dH, dW, bf16=(False, False)):
    """Largest error over its bound, of dH and of dW (at most 1 where they hold)."""
    b = bounds(H, W, y, bf16)
    return tuple(float((np.abs(got - b[k][0]) / b[k][1]).max()) for k, got in (("dH", dH), ("dW", dW)))


def confident(N, D, V, seed, low, high):
    """H, W (fp64 values exact in bf16) and labels: token i's label has a logit of low .. high above the others'.

    The labels' rows of W lie along their tokens, and the other rows are small,
    so that the labels' entries make up most of dH and dW; every label once."""
    rng = np.random.default_rng(seed)
    H = rng.standard_normal((N, D))
    W = 0.01 * rng.standard_normal((V, D))
    y = rng.permutation(V)[:N]
    # tokens nearly orthogonal to one another's label rows
    q, _ = np.linalg.qr(rng.standard_normal((D, D)))
    H = q[np.arange(N) % D] * np.sqrt(D) + 0.01 * H
    t = np.linspace(low, high, N) + np.log(V)
    W[y] = H / D * t[:, None]
    return bf16_values(H), bf16_values(W), y.astype(np.int32)


def bf16_values(x):
    """Rounded to the nearest bf16 value, ties to even."""
    m, e = np.frexp(np.asarray(x, dtype=np.float64))
    return np.ldexp(np.rint(m * 256.0) / 256.0, e)
