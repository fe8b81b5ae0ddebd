"""Outputs in place of inputs, and the largest output layer against 64-bit sums (GPU).

An output may be the very matrix of an input of the same size: the gradients of
the cross-entropy over H and over W, those of the norm over what they come from.
In place the same bits come out as apart.
"""

import pytest
import torch

from layer_optimizer_gb300 import native, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _lce(H, W, y, dH, dW, piece):
    loss, tok = torch.empty(1, device=DEV), torch.empty(H.shape[0], device=DEV)
    ws = torch.empty(native.lce_vocab_workspace_bytes(*H.shape, W.shape[0], piece), dtype=torch.uint8, device=DEV)
    native.lce_vocab_forward_backward(H, W, y, loss=loss, token_loss=tok, dH=dH, dW=dW, ws=ws, piece=piece)
    native.sf_sync_status()
    return loss, tok, dH, dW


@pytest.mark.parametrize("N,D,V,piece", [
    (3, 64, 500, 0), (16, 1032, 9001, 0),               # few tokens
    (17, 64, 500, 0), (300, 136, 2001, 256), (1000, 256, 700, 512),
    (700, 64, 131, 0), (64, 72, 20000, 0),              # sums in parts
    (2100, 520, 5000, 1024),
])
def test_cross_entropy_gradients_over_their_inputs(N, D, V, piece):
    H, W = synth.normal((N, D), 1.0, N, dtype=BF).to(DEV), synth.normal((V, D), 0.05, V, dtype=BF).to(DEV)
    y = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(N), dtype=torch.int32).to(DEV)
    y[:: 5] = -100
    want = _lce(H, W, y, torch.empty_like(H), torch.empty_like(W), piece)
    for over_h, over_w in ((True, False), (False, True), (True, True)):
        h, w = H.clone(), W.clone()
        got = _lce(h, w, y, h if over_h else torch.empty_like(H), w if over_w else torch.empty_like(W), piece)
        for a, b in zip(got, want):
            assert torch.equal(a, b), (over_h, over_w)


@pytest.mark.parametrize("rows,cols", [(5, 264), (64, 2048), (400, 1021), (400, 4096), (330, 4095), (320, 12288)])
@pytest.mark.parametrize("t", [BF, F32])
def test_norm_gradients_over_their_inputs(rows, cols, t):
    dh, s, ds = (synth.normal((rows, cols), 1.0, i, dtype=t).to(DEV) for i in (1, 2, 3))
    gain = (1.0 + synth.normal((cols,), 0.2, 4)).to(DEV)
    rstd = torch.rsqrt(s.double().square().mean(dim=1) + 1e-5).float()
    ws = torch.empty(native.sf_add_rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    dg = torch.empty(cols, device=DEV)

    def run(dh, s, ds, dr, dx):
        native.sf_add_rmsnorm_backward(dh, s, gain, rstd, dsum=ds, dresidual=dr, dx=dx, dgain=dg, p=0.1, rng=native.rng(1, 2), ws=ws)
        native.sf_sync_status()
        return dr, dx, dg.clone()
    want = run(dh, s, ds, torch.empty_like(s), torch.empty_like(dh))
    for pick in (lambda a, b, c: (b, a), lambda a, b, c: (c, a), lambda a, b, c: (c, b), lambda a, b, c: (a, b), lambda a, b, c: (b, c)):
        ins = [v.clone() for v in (dh, s, ds)]
        for a, b in zip(run(*ins, *pick(*ins)), want):
            assert torch.equal(a, b)


def test_largest_output_layer_on_sampled_rows():
    # an 8192-token batch of a 128256-output layer of width 4096, in the default pieces: rows of dH and dW in 64 bits
    N, D, V = 8192, 4096, 128256
    g = torch.Generator(device=DEV).manual_seed(5)
    H = torch.randn(N, D, generator=g, device=DEV).to(BF)
    W = (0.02 * torch.randn(V, D, generator=g, device=DEV)).to(BF)
    y = torch.randint(0, V, (N,), generator=g, device=DEV, dtype=torch.int32)
    y[::10] = -100
    y[3], y[4], y[5] = 0, V - 1, 65535
    loss, tok, dH, dW = _lce(H, W, y, torch.empty_like(H), torch.empty_like(W), 0)
    on = y >= 0
    n = int(on.sum())
    at = y.long().clamp_min(0)[:, None]
    # logits in fp32 (4096 products each: relative 4096 u at the worst, 1e-5 of sum |h||w| taken as everywhere), their sums in 64 bits
    lse, zy = torch.empty(N, dtype=torch.float64, device=DEV), torch.empty(N, dtype=torch.float64, device=DEV)
    assert not torch.backends.cuda.matmul.allow_tf32
    W32 = W.float()
    for i in range(0, N, 1024):
        z = (H[i:i + 1024].float() @ W32.t()).double()
        lse[i:i + 1024] = torch.logsumexp(z, dim=1)
        zy[i:i + 1024] = z.gather(1, at[i:i + 1024])[:, 0]
    z_err = 1e-5 * float(H.float().norm(dim=1).max() * W.float().norm(dim=1).max())      # at least 1e-5 of sum |h||w|
    want = torch.where(on, lse - zy, 0.0)
    assert float((tok.double() - want).abs().max()) <= 4 * z_err + 2e-5
    assert abs(float(loss) - float(want.sum() / n)) <= 4 * z_err + 2e-5

    # dZ: bf16 once or twice (2^-8 each of p), z_err through the exponential and the sum; then bf16 of the result
    def close(got, ref, mag):
        err = (got.double() - ref).abs()
        assert bool((err <= (2 * 2.0 ** -8 + 4 * z_err + 4e-5) * mag + 2.0 ** -8 * ref.abs()).all()), float((err / mag).max())
    del W32
    tokens = [0, 1, 3, 4, 5, 255, 256, 4095, 4096, 8190, 8191]
    W64 = W.double()
    dz = torch.exp(H[tokens].double() @ W64.t() - lse[tokens, None])
    dz[torch.arange(len(tokens)), at[tokens, 0]] -= 1.0
    dz = dz * on[tokens, None] / n
    close(dH[tokens], dz @ W64, dz.abs() @ W64.abs())
    assert not dH[0].any()
    del W64
    outputs = [0, 1, 255, 256, 64127, 64128, 65535, 65536, 128000, V - 1]
    H64 = H.double()
    dz = torch.exp(H64 @ W[outputs].double().t() - lse[:, None])
    dz -= (y[:, None] == torch.tensor(outputs, device=DEV)[None]).double()
    dz = dz * on[:, None] / n
    close(dW[outputs], dz.t() @ H64, dz.abs().t() @ H64.abs())
