"""The label's entry of the vocabulary-piece cross-entropy's gradient (GPU).

Where the model is sure of a label, its entry p - 1 is small and is most of the
token's gradient: it may be rounded once, and not lose p's digits first.
Bounds: _label_entry.py.
"""

import pytest
import torch

from _label_entry import confident, outside
from _util import f64
from layer_optimizer_gb300 import native, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _gradients(H, W, y, t, piece):
    N, D = H.shape
    V = W.shape[0]
    dH, dW, tok = torch.empty(N, D, dtype=t, device=DEV), torch.empty(V, D, dtype=t, device=DEV), torch.empty(N, device=DEV)
    ws = torch.empty(native.lce_vocab_workspace_bytes(N, D, V, piece), dtype=torch.uint8, device=DEV)
    native.lce_vocab_forward_backward(H, W, y, token_loss=tok, dH=dH, dW=dW, ws=ws, piece=piece)
    native.sf_sync_status()
    return dH, dW, tok


@pytest.mark.parametrize("N,D,V,piece", [(16, 64, 600, 0), (5, 64, 1030, 0), (48, 64, 1030, 0), (48, 64, 1030, 256), (48, 64, 600, 512),
                                         (17, 72, 300, 256)])
@pytest.mark.parametrize("low,high", [(1.0, 6.0), (3.0, 5.0)])
@pytest.mark.parametrize("t", [F32, BF])
def test_confident_tokens(N, D, V, piece, low, high, t):
    H, W, y = confident(N, D, V, N + V, low, high)
    dev = [torch.from_numpy(a).to(BF).to(DEV) for a in (H, W)]
    dH, dW, _ = _gradients(*dev, torch.from_numpy(y).to(DEV), t, piece)
    assert max(outside(H, W, y, f64(dH.float()), f64(dW.float()), (t == BF, t == BF))) <= 1.0


@pytest.mark.parametrize("label", [3, 300, 1029])
def test_the_entry_does_not_depend_on_the_piece(label):
    # one labelled token: dW's row of its label is the entry times the token's row of H
    N, D, V = 20, 64, 1030
    H = synth.normal((N, D), 1.0, 1, dtype=BF)
    h = H[7].float()
    y = torch.full((N,), -100, dtype=torch.int32, device=DEV)
    y[7] = label
    for k in range(40):
        # logits of 8 to 20 against some thousand outputs near 0: 1 - p from 0.3 down to 1e-6
        W = synth.normal((V, D), 0.01, 2 + k, dtype=BF)
        W[label] = (h * ((8.0 + 0.3 * k) / float(h @ h))).to(BF)
        rows = [_gradients(H.to(DEV), W.to(DEV), y, F32, piece) for piece in (0, 256, 512, 1024)]
        for dH, dW, tok in rows[1:]:
            assert torch.equal(tok, rows[0][2])
            assert torch.equal(dW[label], rows[0][1][label]), (k, float(tok[7]))
