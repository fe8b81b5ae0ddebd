"""Linear cross-entropy by pieces of the vocabulary against the fp64 oracle (GPU).

Tolerances, derived from the arithmetic:

* logits: bf16 products summed in fp32 on the tensor cores, within
  z_err = 1e-5 of sum |h||w| (the library's bound for its GEMM).
* a token's loss: two logits, and the log-sum-exp's own error: chains of at
  most 8 + 8 + n_tiles / 32 + 7 additions of positive terms and the
  exponential's 2^-22 (8e-6 taken), logf and the difference 4u of |lse|.
* dZ = (p - onehot) / n: p relative within 2 z_err + 1e-5; the entry rounded to
  bf16 once (2^-8 of it), the last piece's twice (the exponential first: 2^-8
  of p more).  dH and dW: those errors through |W| and |H|, 1e-5 of
  |dZ||W| and |dZ|^T|H| for the sums, and half a unit in the last place
  where stored in bf16.
"""

import numpy as np
import pytest
import torch

from _util import f64
from layer_optimizer_gb300 import native, synth
from oracle.lce import lce

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _case(N, D, V, seed, unlabelled=0, hstd=1.0, wstd=0.02):
    H = synth.normal((N, D), hstd, seed, dtype=BF)
    W = synth.normal((V, D), wstd, seed + 1, dtype=BF)
    g = torch.Generator().manual_seed(seed + 2)
    y = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    if unlabelled:
        y[torch.randperm(N, generator=g)[:unlabelled]] = -100
    return H, W, y


def _dev(t, pad=0):
    """On the device, rows `pad` elements apart from dense; the padding holds NaN."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=DEV)
    v = buf[:, :t.shape[1]]
    v.copy_(t)
    return v


def _run(H, W, y, piece=0, ht=BF, wt=BF, pad=0, opad=0, dh=True, dw=True, grad_scale=1.0, stream=None):
    N, D = H.shape
    V = W.shape[0]
    Hd, Wd = (t if t.is_cuda else _dev(t, pad) for t in (H, W))
    wsb = native.lce_vocab_workspace_bytes(N, D, V, piece)
    ws = torch.full((wsb + 256,), 0xFF, dtype=torch.uint8, device=DEV)     # NaN everywhere, and a guard behind
    loss, tok = torch.full((1,), float("nan"), device=DEV), torch.full((N,), float("nan"), device=DEV)
    hb = torch.full((N + 1, D + opad), 7.0, dtype=ht, device=DEV)
    wb = torch.full((V + 1, D + opad), 7.0, dtype=wt, device=DEV)
    dH, dW = hb[:N, :D], wb[:V, :D]
    torch.cuda.synchronize()
    native.lce_vocab_forward_backward(Hd, Wd, y.to(DEV), loss=loss, token_loss=tok, dH=dH if dh else None,
                                      dW=dW if dw else None, ws=ws[:wsb], piece=piece, grad_scale=grad_scale, stream=stream)
    native.sf_sync_status(stream)
    assert bool((ws[wsb:] == 0xFF).all()), "workspace guard"
    for b, n in ((hb, N), (wb, V)):
        assert bool((b[n:] == 7.0).all()) and bool((b[:, D:] == 7.0).all()), "output guard"
    if not dh:
        assert bool((hb == 7.0).all())
    if not dw:
        assert bool((wb == 7.0).all())
    return loss, tok, dH, dW


def _half_ulp(x, dtype):
    _, e = np.frexp(x)
    return np.ldexp(0.5, e - (8 if dtype == BF else 24))


def _check(H, W, y, got, grad_scale=1.0):
    loss, tok, dH, dW = got
    H64, W64, yn = f64(H.float()), f64(W.float()), y.cpu().numpy()
    V = W64.shape[0]
    on = (yn >= 0) & (yn < V)
    res = lce(H64, W64, np.where(on, yn, -100))
    n = max(1, res["n"])
    z_err = 1e-5 * (np.abs(H64) @ np.abs(W64).T)
    want = np.where(on, res["lse"] - res["Z"][np.arange(len(yn)), np.where(on, yn, 0)], 0.0)
    bound = np.where(on, 2 * z_err.max(axis=1) + 8e-6 + 4 * U * np.abs(res["lse"]), 0.0)
    err = np.abs(f64(tok) - want)
    assert (err <= bound).all(), ("token_loss", float((err / np.maximum(bound, 1e-300)).max()))
    assert abs(float(loss) - res["loss"]) <= bound.sum() / n + 2 * U * abs(res["loss"])
    P = np.exp(res["Z"] - res["lse"][:, None]) * on[:, None] / n
    eZ = P * (2 * z_err.max() + 1e-5 + 2.0 ** -8) + np.abs(res["dZ"]) * (2.0 ** -8 + 1e-5)
    for name, out, ref, err_z in (("dH", dH, res["dH"], eZ @ np.abs(W64)), ("dW", dW, res["dW"], eZ.T @ np.abs(H64))):
        ref, err_z = ref * grad_scale, err_z * abs(grad_scale)
        err = np.abs(f64(out.float()) - ref)
        b = err_z + _half_ulp(np.abs(ref) + err_z, out.dtype) + 1e-38
        assert (err <= b).all(), (name, int((err > b).sum()), float((err / b).max()))
    return res


@pytest.mark.parametrize("N,D,V,piece,unlabelled", [
    (1, 8, 1, 0, 0),                # one class: loss 0, no gradient
    (1, 64, 1000, 0, 0),            # one token
    (1, 1024, 5003, 256, 0),        # one token, twenty pieces
    (7, 24, 257, 256, 2),           # a last piece of one column
    (300, 64, 521, 256, 20),
    (129, 96, 2048, 512, 0),
    (1000, 256, 1001, 0, 100),
    (257, 512, 3333, 1024, 1),
    (64, 72, 40000, 0, 8),          # few tokens, long vocabulary: dH's sum in parts
    (2048, 64, 300, 0, 64),         # many tokens, few outputs: dW's sum in parts
    (40, 32, 264, 0, 40),           # every token unlabelled
    (8200, 16, 8200, 0, 70),        # short rows and many logits: the last piece's computed twice as well
])
def test_matches_oracle(N, D, V, piece, unlabelled):
    H, W, y = _case(N, D, V, N + D + V, unlabelled)
    _check(H, W, y, _run(H, W, y, piece))


@pytest.mark.parametrize("ht,wt,pad,opad,D", [(F32, F32, 0, 0, 64), (F32, BF, 8, 8, 64), (BF, F32, 16, 4, 60), (BF, BF, 3, 3, 61),
                                              (F32, F32, 7, 3, 65)])
@pytest.mark.parametrize("N,V,piece", [(200, 1111, 512), (70, 700, 0)])
def test_output_types_strides_and_odd_widths(ht, wt, pad, opad, D, N, V, piece):
    H, W, y = _case(N, D, V, 5 + D, 9)
    pad, opad = -(D + pad) % 8 + pad, -(D + opad) % 8 + opad      # rows of 16-byte multiples around D columns
    _check(H, W, y, _run(H, W, y, piece, ht, wt, pad, opad))


@pytest.mark.parametrize("N,D,V,unlabelled", [
    (16, 8, 5, 0), (2, 32, 33, 0), (9, 40, 4099, 3), (16, 72, 2500, 4), (13, 136, 1000, 0), (5, 264, 70, 1), (3, 520, 777, 0),
    (16, 1096, 3001, 15), (1, 4096, 600, 0), (16, 64, 12345, 16), (8, 2048, 130, 0),
])
@pytest.mark.parametrize("ht,wt,pad,opad", [(BF, BF, 0, 0), (F32, F32, 8, 8), (BF, F32, 16, 24), (F32, BF, 0, 8)])
def test_few_tokens(N, D, V, unlabelled, ht, wt, pad, opad):
    H, W, y = _case(N, D, V, N + D + V, unlabelled)
    got = _run(H, W, y, 0, ht, wt, pad, opad)
    _check(H, W, y, got)
    off = y == -100
    bad = H.clone()
    bad[off] = float("nan")
    for a, b in zip(got, _run(bad, W, y, 0, ht, wt, pad, opad)):
        assert torch.equal(a, b)
    only_h, only_w, none = (_run(H, W, y, 0, ht, wt, dh=d, dw=w) for d, w in ((True, False), (False, True), (False, False)))
    assert torch.equal(only_h[2], got[2]) and torch.equal(only_w[3], got[3])
    for r in (only_h, only_w, none):
        assert torch.equal(r[0], got[0]) and torch.equal(r[1], got[1])
    _check(H, W, y, _run(H, W, y, 0, ht, wt, pad, opad, grad_scale=-3.0), -3.0)


@pytest.mark.parametrize("N", [3, 40])
def test_outputs_that_are_all_nan_reach_every_loss(N):
    # a run of vocabulary rows long enough to fill whole tiles
    H, W, y = _case(N, 64, 2000, 77)
    W[512:1100] = float("nan")
    for piece in (0, 1024):
        loss, tok, dH, _ = _run(H, W, y, piece)
        assert bool(torch.isnan(loss).all()) and bool(torch.isnan(tok).all()) and bool(torch.isnan(dH.float()).all())


def test_large_and_confident_logits():
    # logits of several hundred: exponentials of raw logits would overflow
    H, W, y = _case(100, 64, 600, 3, 4, hstd=8.0, wstd=2.0)
    _check(H, W, y, _run(H, W, y, 256))
    # the label's probability close to 1 in every piece: its entry p - 1 must not be lost to rounding
    H, W, y = _case(300, 64, 600, 4)
    H = (W[y.long()].float() * 400).to(BF)
    for piece in (0, 256):
        _check(H, W, y, _run(H, W, y, piece))


def test_labels_at_piece_and_tile_edges():
    N, D, V = 16, 64, 1030
    H, W, _ = _case(N, D, V, 8)
    y = torch.tensor([0, 1, 255, 256, 257, 511, 512, 767, 768, 1023, 1024, 1029, 31, 32, 63, 64], dtype=torch.int32)
    for piece in (256, 512, 1024, 0):
        _check(H, W, y, _run(H, W, y, piece))


def test_unlabelled_ids_and_bad_labels():
    N, D, V = 64, 64, 300
    H, W, y = _case(N, D, V, 12, 10)
    res = _check(H, W, y, _run(H, W, y))
    assert res["n"] == N - 10
    got = _run(H, W, y)
    off = (y == -100).to(DEV)
    assert not got[2][off].any() and not got[1][off].any()
    # a label beyond the vocabulary counts as unlabelled and is reported
    bad = y.clone()
    bad[3], bad[5], bad[7] = V, -7, 2 ** 31 - 1
    ws = torch.empty(native.lce_vocab_workspace_bytes(N, D, V), dtype=torch.uint8, device=DEV)
    out = (torch.empty(1, device=DEV), torch.empty(N, device=DEV), torch.empty(N, D, device=DEV), torch.empty(V, D, device=DEV))
    native.lce_vocab_forward_backward(H.to(DEV), W.to(DEV), bad.to(DEV), loss=out[0], token_loss=out[1], dH=out[2], dW=out[3],
                                      ws=ws)
    with pytest.raises(native.SfError, match="out-of-range"):
        native.sf_sync_status()
    _check(H, W, bad, out)


def _run_prepared(H, W, y, piece):
    N, D, V = H.shape[0], H.shape[1], W.shape[0]
    wsb = native.lce_vocab_workspace_bytes(N, D, V, piece)
    ws = torch.full((wsb,), 0xFF, dtype=torch.uint8, device=DEV)
    out = (torch.empty(1, device=DEV), torch.empty(N, device=DEV), torch.empty(N, D, dtype=BF, device=DEV),
           torch.empty(V, D, dtype=BF, device=DEV))
    native.lce_vocab_forward_backward(H.to(DEV), W.to(DEV), y.to(DEV), loss=out[0], token_loss=out[1], dH=out[2], dW=out[3],
                                      ws=ws, piece=piece)
    native.sf_sync_status()
    return out


@pytest.mark.parametrize("N,labelled", [(1000, 1), (1000, 64), (1000, 65), (1000, 97), (1000, 257), (513, 512), (70, 70)])
@pytest.mark.parametrize("piece", [0, 256])
def test_mostly_unlabelled_tokens(N, labelled, piece):
    # prompts masked out: the labelled tokens alone count, wherever they stand; what the others hold reaches nothing
    D, V = 72, 700
    H, W, y = _case(N, D, V, labelled + N, N - labelled)
    clean = _run_prepared(H, W, y, piece)
    _check(H, W, y, clean)
    off = y == -100
    bad = H.clone()
    bad[off] = float("nan")
    bad[off.nonzero()[::2, 0]] = float("inf")
    for a, b in zip(clean, _run_prepared(bad, W, y, piece)):
        assert torch.equal(a, b)


def test_outputs_left_out_grad_scale_and_repeatability():
    H, W, y = _case(300, 128, 1500, 21, 30)
    full = _run(H, W, y, 512)
    again = _run(H, W, y, 512)
    for a, b in zip(full, again):
        assert torch.equal(a, b)
    only_h, only_w, none = _run(H, W, y, 512, dw=False), _run(H, W, y, 512, dh=False), _run(H, W, y, 512, dh=False, dw=False)
    assert torch.equal(only_h[2], full[2]) and torch.equal(only_w[3], full[3])
    for r in (only_h, only_w, none):
        assert torch.equal(r[0], full[0]) and torch.equal(r[1], full[1])
    _check(H, W, y, _run(H, W, y, 512, grad_scale=-0.125), -0.125)
    # the losses do not depend on the pieces
    whole = _run(H, W, y, 0)
    assert torch.equal(whole[0], full[0]) and torch.equal(whole[1], full[1])


def test_agrees_with_the_token_chunk_form():
    N, D, V = 1000, 256, 4000
    H, W, y = _case(N, D, V, 31, 50)
    loss, tok, dH, dW = _run(H, W, y, 1024, F32, F32)
    wsb = native.lce_workspace_bytes(N, D, V, 256)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    l2, h2, w2 = torch.empty(1, dtype=torch.float64, device=DEV), torch.empty(N, D, device=DEV), torch.empty(V, D, device=DEV)
    native.lce_forward_backward(H.to(DEV), W.to(DEV), y.to(DEV), N, D, V, 256, -100, l2, h2, w2, ws, wsb)
    native.sf_sync_status()
    # both round dZ to bf16 (2^-8 of it at most, in the worst direction in each)
    assert abs(float(loss) - float(l2)) <= 1e-5 * float(l2)
    assert float((dH - h2).norm() / h2.norm()) < 2.0 ** -7 and float((dW - w2).norm() / w2.norm()) < 2.0 ** -7


def test_on_another_stream_and_in_a_graph():
    N, D, V = 200, 128, 1000
    H, W, y = _case(N, D, V, 41)
    want = _run(H, W, y, 256)
    st = torch.cuda.Stream()
    for a, b in zip(want, _run(H, W, y, 256, stream=st)):
        assert torch.equal(a, b)
    Hd, Wd, yd = H.to(DEV), W.to(DEV), y.to(DEV)
    ws = torch.empty(native.lce_vocab_workspace_bytes(N, D, V, 256), dtype=torch.uint8, device=DEV)
    out = [torch.zeros_like(t) for t in want]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        native.lce_vocab_forward_backward(Hd, Wd, yd, loss=out[0], token_loss=out[1], dH=out[2], dW=out[3], ws=ws, piece=256,
                                          stream=torch.cuda.current_stream())
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b)
        for t in out:
            t.zero_()


def test_refusals():
    H, W, y = _case(64, 64, 300, 1)
    Hd, Wd, yd = H.to(DEV), W.to(DEV), y.to(DEV)
    ws = torch.empty(native.lce_vocab_workspace_bytes(64, 64, 300), dtype=torch.uint8, device=DEV)
    dH, dW = torch.empty(64, 64, device=DEV), torch.empty(300, 64, device=DEV)

    def call(match, H=Hd, W=Wd, y=yd, **kw):
        with pytest.raises(native.SfError, match=match):
            native.lce_vocab_forward_backward(H, W, y, **{**dict(ws=ws, dH=dH, dW=dW), **kw})

    call("workspace", ws=ws[:-256])
    call("workspace", ws=ws[16:])
    call("workspace", ws=None)
    call("multiple of 256", piece=100)
    call("multiple of 256", piece=-256)
    call("finite", grad_scale=float("inf"))
    call("expected", W=Wd[:, :56])
    call("not taken", H=Hd.float())
    call("16-byte", H=torch.empty(64, 65, dtype=BF, device=DEV)[:, 1:])
    call("16-byte", W=torch.empty(300, 68, dtype=BF, device=DEV)[:, :64])
    call("16-byte", dW=torch.empty(300, 65, device=DEV)[:, :64])
    call("expected", dH=dW)
    call("labels", y=None)
    call("dense with 64", y=yd[:10])
    call("not taken", y=yd.long())
    call("at least one", H=Hd[:0], y=yd[:0], dH=dH[:0])
    native.sf_sync_status()
