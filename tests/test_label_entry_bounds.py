"""The bounds on the label's entry catch the mistakes that they name (CPU only)."""

import numpy as np
import pytest

from _label_entry import bf16_values, confident, outside
from oracle.lce import lce

# (few tokens, and more) times (labels in every piece of 256 outputs)
CASES = [(16, 64, 600, 1), (48, 64, 1030, 2)]


def _gradients(H, W, y, entry):
    """dH and dW of dZ in bf16, the label's entry from entry(p, p - 1)."""
    res = lce(H, W, y)
    rows = np.arange(len(y))
    P = np.exp(res["Z"] - res["lse"][:, None])
    G = bf16_values(bf16_values(P))
    G[rows, y] = entry(P[rows, y], np.expm1((res["Z"] - res["lse"][:, None])[rows, y]))
    G = G / len(y)
    return G @ W, G.T @ H


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("low,high", [(1.0, 6.0), (3.0, 5.0)])
def test_the_entry_rounded_once_holds(case, low, high):
    H, W, y = confident(*case, low, high)
    assert max(outside(H, W, y, *_gradients(H, W, y, lambda p, m: bf16_values(m)))) <= 1.0


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("low,high", [(1.0, 6.0), (3.0, 5.0)])
@pytest.mark.parametrize("mistake", [
    lambda p, m: bf16_values(bf16_values(p) - 1.0),      # rounded before 1 is taken off
    lambda p, m: bf16_values(p),                         # nothing taken off
    lambda p, m: 0.0 * m,                                # no gradient at the label
])
def test_planted_mistakes_at_the_label_fail(case, low, high, mistake):
    H, W, y = confident(*case, low, high)
    dh, dw = outside(H, W, y, *_gradients(H, W, y, mistake))
    assert dh > 1.0 and dw > 1.0
