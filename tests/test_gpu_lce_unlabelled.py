"""Unlabelled tokens of the vocabulary-piece cross-entropy, whatever the weights hold (GPU).

A token without a label has no loss and no gradient: exactly 0, at every number
of tokens, also where W holds NaN or infinities and where no token has a label
at all.
"""

import pytest
import torch

from layer_optimizer_gb300 import native, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _run(H, W, y, ht, wt, piece=0):
    N, D = H.shape
    V = W.shape[0]
    full = lambda shape, t: torch.full(shape, float("nan"), dtype=t, device=DEV)  # noqa: E731
    width = D + -D % 8      # rows of whole 16-byte units
    loss, tok, dH, dW = full((1,), F32), full((N,), F32), full((N, width), ht)[:, :D], full((V, width), wt)[:, :D]
    ws = torch.full((native.lce_vocab_workspace_bytes(N, D, V, piece),), 0xFF, dtype=torch.uint8, device=DEV)
    native.lce_vocab_forward_backward(H, W, y, loss=loss, token_loss=tok, dH=dH, dW=dW, ws=ws, piece=piece)
    native.sf_sync_status()
    return loss, tok, dH, dW


@pytest.mark.parametrize("N,D,V,piece", [(1, 64, 300, 0), (7, 8, 33, 0), (16, 520, 5000, 0), (16, 1032, 40000, 0), (17, 520, 5000, 0),
                                         (40, 64, 700, 256), (9, 61, 700, 0), (300, 72, 1030, 512)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ht,wt", [(BF, BF), (F32, F32)])
def test_weights_that_are_not_finite_reach_no_unlabelled_token(N, D, V, piece, bad, ht, wt):
    pad = -D % 8
    H = synth.normal((N, D + pad), 1.0, N + D, dtype=BF).to(DEV)[:, :D]
    W = synth.normal((V, D + pad), 0.02, V, dtype=BF).to(DEV)[:, :D]
    y = torch.arange(N, dtype=torch.int32, device=DEV) % V
    y[::2] = -100
    W[V // 2] = bad
    W[-1, 0] = bad
    _, tok, dH, _ = _run(H, W, y, ht, wt, piece)
    assert not tok[::2].any() and not dH[::2].any()
    if bad != bad:      # every labelled token's logits hold a NaN
        assert bool(torch.isnan(tok[1::2]).all()) and bool(torch.isnan(dH[1::2].float()).all())
    # no label at all: no loss, no gradient
    y.fill_(-100)
    for out in _run(H, W, y, ht, wt, piece):
        assert not out.any()
