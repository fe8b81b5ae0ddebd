"""Offsets past 2^31 elements, and host memory, for the output end's operators (GPU).

Big cases are checked on sampled rows: a row of a norm or of a dropout depends
on itself (and its index) alone, so the same rows in a small call, or the fp64
oracle of those rows, are the reference.
"""

import numpy as np
import pytest
import torch

from _util import f64
from layer_optimizer_gb300 import native, synth
from oracle import dropout as od
from oracle import norm as on

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
ROWS, COLS = 530001, 4096            # 2.17e9 elements
PICK = [0, 1, 262143, 262144, 524287, 524288, 524289, ROWS - 1]


def _mask_rows(rows, cols, p, seed, offset):
    """The kept elements of single rows, counter by counter."""
    out = np.empty((len(rows), cols), dtype=bool)
    per = -(-cols // 8)
    for i, r in enumerate(rows):
        for u in range(per):
            b = r * per + u
            w = od.philox4x32((b & od.LOW, b >> 32, offset & od.LOW, offset >> 32), (seed & od.LOW, seed >> 32))
            for c in range(8 * u, min(cols, 8 * u + 8)):
                word = w[(c % 8) // 2]
                out[i, c] = (word & 0xFFFF if c % 2 == 0 else word >> 16) >= od.threshold(p)
    return out


@pytest.fixture(scope="module")
def big():
    x = torch.empty(ROWS, COLS, dtype=BF, device=DEV)
    synth.fill_normal_(x, 1.0, 5)
    return x


def test_dropout_past_2_31(big):
    y = torch.full_like(big, 7.0)
    native.sf_dropout(big, y, 0.5, native.rng(9, 1 << 33))
    native.sf_sync_status()
    got, x = y[PICK].float().cpu().numpy(), big[PICK].float().cpu().numpy()
    kept = _mask_rows(PICK, COLS, 0.5, 9, 1 << 33)
    assert np.array_equal(got, np.where(kept, 2.0 * x, 0.0))        # the factor is 2: exact in bf16


def test_norm_past_2_31(big):
    gain = (1.0 + synth.normal((COLS,), 0.1, 6)).to(DEV)
    s, h, rstd = torch.empty_like(big), torch.empty_like(big), torch.empty(ROWS, device=DEV)
    native.sf_add_rmsnorm_forward(big, big, gain, 1e-5, sum=s, h=h, rstd=rstd)
    native.sf_sync_status()
    few = big[PICK].contiguous()
    s2, h2, r2 = torch.empty_like(few), torch.empty_like(few), torch.empty(len(PICK), device=DEV)
    native.sf_add_rmsnorm_forward(few, few, gain, 1e-5, sum=s2, h=h2, rstd=r2)
    assert torch.equal(s[PICK], s2)
    ref, rr = on.forward(2.0 * f64(few.float()), f64(gain), 1e-5)
    for got in (h[PICK], h2):
        # half a unit in bf16's last place, and the fp32 error below it
        assert np.all(np.abs(f64(got.float()) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-30)
    assert np.all(np.abs(f64(rstd[PICK]) - rr) <= 1e-5 * rr)
    # backward in place: h is the gradient, the sum's gradient lands on s
    ds, _, mag, _ = on.backward(f64(h[PICK].float()), f64(s[PICK].float()), f64(gain), 1e-5)
    r3 = torch.rsqrt(s[PICK].double().square().mean(dim=1) + 1e-5).float()
    rstd[PICK] = r3
    native.sf_add_rmsnorm_backward(h, s, gain, rstd, dresidual=s, dx=h)
    native.sf_sync_status()
    for got in (s[PICK], h[PICK]):
        assert np.all(np.abs(f64(got.float()) - ds) <= 2.0 ** -8 * np.abs(ds) + 1e-5 * mag)


def test_vocabulary_past_2_31():
    N, D, V = 5, COLS, ROWS
    W = torch.empty(V, D, dtype=BF, device=DEV)
    synth.fill_normal_(W, 0.02, 8)
    H = synth.normal((N, D), 1.0, 9, dtype=BF).to(DEV)
    y = torch.tensor([0, 524288, V - 1, -100, V // 2], dtype=torch.int32, device=DEV)
    dH, dW = torch.empty_like(H), torch.full_like(W, 7.0)
    tok = torch.empty(N, device=DEV)
    ws = torch.empty(native.lce_vocab_workspace_bytes(N, D, V, 65536), dtype=torch.uint8, device=DEV)
    native.lce_vocab_forward_backward(H, W, y, token_loss=tok, dH=dH, dW=dW, ws=ws, piece=65536)
    native.sf_sync_status()
    H64 = H.double()
    z = torch.cat([H64 @ W[v:v + 16384].double().t() for v in range(0, V, 16384)], dim=1)
    lse = torch.logsumexp(z, dim=1)
    on_ = y >= 0
    want = torch.where(on_, lse - z.gather(1, y.long().clamp_min(0)[:, None])[:, 0], 0.0)
    z_err = 1e-5 * float(H64.abs().sum(dim=1).max()) * 0.12          # |w| <= 6 standard deviations
    assert float((tok.double() - want).abs().max()) <= 2 * z_err + 2e-5
    dz = torch.exp(z - lse[:, None])
    dz[on_, y[on_].long()] -= 1.0
    dz = dz * on_[:, None] / 4
    pick = [0, 1, 65535, 65536, 524287, 524288, V - 2, V - 1]
    ref = dz[:, pick].t() @ H64
    mag = dz[:, pick].abs().t() @ H64.abs()
    assert bool(((dW[pick].double() - ref).abs() <= (2.0 ** -7 + 2 * z_err) * mag + 2.0 ** -8 * ref.abs()).all())
    rh = torch.zeros_like(H64)
    rm = torch.zeros_like(H64)
    for v in range(0, V, 16384):
        w = W[v:v + 16384].double()
        rh += dz[:, v:v + 16384] @ w
        rm += dz[:, v:v + 16384].abs() @ w.abs()
    assert bool(((dH.double() - rh).abs() <= (2.0 ** -7 + 2 * z_err) * rm + 2.0 ** -8 * rh.abs()).all())
    assert not dH[3].any()


def test_pinned_host_rows_give_the_device_results():
    rows, cols = 400, 1024
    host = [synth.normal((rows, cols), 1.0, 20 + i, dtype=BF).pin_memory() for i in range(3)]
    outs = [torch.zeros(rows, cols, dtype=BF).pin_memory() for _ in range(2)]
    gain = torch.ones(cols, dtype=BF, device=DEV)
    rstd = torch.rand(rows, device=DEV) + 0.5
    dev, dout = [t.to(DEV) for t in host], [torch.empty(rows, cols, dtype=BF, device=DEV) for _ in range(2)]
    rng = native.rng(1, 2)
    for (a, b, c), (o, q) in ((host, outs), (dev, dout)):
        native.sf_add_rmsnorm_backward(a, b, gain, rstd, dsum=c, dresidual=o, dx=q, p=0.25, rng=rng)
    native.sf_sync_status()
    for o, d in zip(outs, dout):
        # the two paths sum a row in different orders: equal up to a last place where the sum's last bit turns a rounding
        assert float((o.float() - d.cpu().float()).abs().max()) <= 2.0 ** -8 * float(d.float().abs().max())
    for (a, b, c), (o, q) in ((host, outs), (dev, dout)):
        native.sf_add_rmsnorm_forward(a, b, gain, 1e-5, sum=o, h=q, p=0.25, rng=rng)
    native.sf_sync_status()
    assert all(torch.equal(o, d.cpu()) for o, d in zip(outs, dout))
    native.sf_dropout(host[0], outs[0], 0.25, rng, residual=host[1])
    native.sf_dropout(dev[0], dout[0], 0.25, rng, residual=dev[1])
    native.sf_sync_status()
    assert torch.equal(outs[0], dout[0].cpu())
    # the cross-entropy reads through tensor maps: host memory is refused
    ws = torch.empty(native.lce_vocab_workspace_bytes(rows, cols, rows), dtype=torch.uint8, device=DEV)
    y = torch.zeros(rows, dtype=torch.int32, device=DEV)
    with pytest.raises(native.SfError, match="device memory"):
        native.lce_vocab_forward_backward(host[0], dev[1], y, dW=dout[0], ws=ws)
