"""Weight gradients from 8-bit checkpoints against the fp64 oracle (GPU).

Products of bf16 values are exact in fp32.  Within a span of 512 tokens the tensor cores add groups of at least 16
products and cut what does not fit their accumulator: 32 steps, each off by at most 2^-22 of the magnitudes so far
(2^-23 cut, doubled for the group's own alignment): 32 2^-22 of the span's magnitudes, 8e-6; spans are joined in fp32,
rounded to nearest: 1e-5 in all.  A product on the CUDA cores adds its tokens one by one: tokens u where that is more.
fp32 scales that are no
powers of two round value * scale to bf16: half a step, 2^-8 of the term at most.
"""

import numpy as np
import pytest
import torch

from _block_end import BF, DEV, E4, F32, close, guard_ok, make_checkpoint, rows_of, stored
from _util import f64
from layer_optimizer_gb300 import native, synth
from oracle import checkpoint as oc

pytestmark = pytest.mark.gpu


def _sum(tokens):
    return max(1e-5, tokens * 2.0 ** -24)


def _run(tokens, out, cin, group, dt, acc, pad=0, lead=0, seed=0, in_place=False):
    dy, _ = rows_of(tokens, out, pad, BF, 51 + seed + tokens, 1e-2, lead)
    x, _ = rows_of(tokens, cin, pad, BF, 52 + seed + tokens, 2.0, lead)
    ck, q, scale = make_checkpoint(x, group, pad, lead)
    dw, buf = rows_of(out, cin, pad, dt, None, lead=lead)
    base = None
    if acc:
        base, _ = rows_of(out, cin, pad, dt, 53 + seed, 0.5, lead)
        if in_place:
            dw.copy_(base)
            kept, base = f64(base.float()), dw
        else:
            kept = f64(base.float())
    ws = torch.empty(max(16, native.sf_checkpoint_wgrad_workspace_bytes(tokens, out, cin)), dtype=torch.uint8, device=DEV)
    native.sf_checkpoint_wgrad(dy, ck, dw, base=base, ws=ws)
    native.sf_sync_status()
    ref, mag = oc.weight_grad(f64(dy.float()), oc.restore(f64(q.float()), f64(scale.float()).reshape(tokens, -1), group), kept if acc else None)
    close("dw", dw, ref, stored(dt, ref, _sum(tokens) * mag))
    assert guard_ok(dw, buf, lead)


TOKENS_OUT_IN = [(1, 8, 16), (1, 1000, 4096), (7, 24, 48), (63, 128, 128), (64, 256, 256), (65, 264, 272), (200, 1000, 1008), (511, 256, 512),
                 (512, 264, 256), (513, 512, 128), (1003, 1000, 1024), (2048, 256, 256), (2100, 40, 5008), (1500, 2000, 640),
                 (1030, 2600, 2048)]      # 88 tiles: a whole wave of pairs and 12 that are split


@pytest.mark.parametrize("tokens,out,cin", TOKENS_OUT_IN)
@pytest.mark.parametrize("group,dt,acc", [(32, BF, False), (128, F32, True), (0, F32, False), (64, BF, True)])
def test_matches_oracle(tokens, out, cin, group, dt, acc):
    _run(tokens, out, cin, group, dt, acc)


# rows that do not start on 16 bytes, a base off them, sizes off every unit
@pytest.mark.parametrize("tokens,out,cin,pad,lead", [(37, 61, 129, 0, 0), (130, 64, 64, 3, 0), (100, 72, 144, 0, 1), (1, 1, 1, 0, 0), (70, 1, 300, 0, 0),
                                                     (70, 300, 1, 0, 0), (600, 130, 257, 6, 0)])
@pytest.mark.parametrize("group,dt,acc", [(32, BF, False), (0, F32, True)])
def test_any_alignment(tokens, out, cin, pad, lead, group, dt, acc):
    _run(tokens, out, cin, group, dt, acc, pad, lead)


@pytest.mark.parametrize("tokens,out,cin", [(100, 264, 272), (1003, 1000, 1024), (37, 61, 129)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_adds_in_place(tokens, out, cin, dt):
    _run(tokens, out, cin, 32, dt, True, in_place=True)


# outputs whose rows end inside 16 bytes, or start off them, next to aligned operands
@pytest.mark.parametrize("dt,cols,pad,lead", [(F32, 272, 1, 0), (BF, 272, 3, 0), (F32, 272, 0, 1), (BF, 272, 8, 2), (BF, 264, 8, 0), (F32, 270, 2, 0),
                                              (BF, 270, 2, 0)])
@pytest.mark.parametrize("acc", [False, True])
def test_outputs_of_every_alignment(dt, cols, pad, lead, acc):
    tokens, out = 300, 300
    dy = rows_of(tokens, out, 4, BF, 61, 1.0)[0]
    wide = -(-cols // 16) * 16
    x = rows_of(tokens, wide, 0, BF, 62, 1.0)[0]
    ck, q, scale = make_checkpoint(x[:, :cols], 64, wide - cols)
    dw, buf = rows_of(out, cols, pad, dt, None, lead=lead)
    base = rows_of(out, cols, pad, dt, 63, 1.0, lead)[0] if acc else None
    ws = torch.empty(max(16, native.sf_checkpoint_wgrad_workspace_bytes(tokens, out, cols)), dtype=torch.uint8, device=DEV)
    native.sf_checkpoint_wgrad(dy, ck, dw, base=base, ws=ws)
    native.sf_sync_status()
    ref, mag = oc.weight_grad(f64(dy.float()), oc.restore(f64(q.float()), f64(scale.float()), 64), None if base is None else f64(base.float()))
    close("dw", dw, ref, stored(dt, ref, _sum(tokens) * mag))
    assert guard_ok(dw, buf, lead)


@pytest.mark.parametrize("cin", [256, 250])
@pytest.mark.parametrize("group", [0, 32])
def test_fp32_scales(cin, group):
    # as the norm's 8-bit output has them: value * scale rounds to bf16, 2^-8 / 2 of a term either way
    tokens, out = 130, 264
    h8 = synth.normal((tokens, cin), 50.0, 71).clamp(-448, 448).to(DEV).to(E4)
    scale = torch.rand(tokens, -(-cin // group) if group else 1, device=DEV) + 0.1
    dy = synth.normal((tokens, out), 1.0, 72).to(BF).to(DEV)
    dw = torch.empty(out, cin, device=DEV)
    ws = torch.empty(max(16, native.sf_checkpoint_wgrad_workspace_bytes(tokens, out, cin)), dtype=torch.uint8, device=DEV)
    native.sf_checkpoint_wgrad(dy, native.checkpoint(h8, scale, group), dw, ws=ws)
    native.sf_sync_status()
    ref, mag = oc.weight_grad(f64(dy.float()), oc.restore(f64(h8.float()), f64(scale), group))
    close("dw", dw, ref, (2.0 ** -8 + _sum(tokens)) * mag)


def test_operands_in_pinned_host_memory():
    tokens, out, cin = 100, 64, 96
    dy = synth.normal((tokens, out), 1.0, 73).to(BF).pin_memory()
    ck, q, scale = make_checkpoint(synth.normal((tokens, cin), 1.0, 74).to(BF).to(DEV), 32)
    hq, hs = q.cpu().pin_memory(), scale.view(torch.uint8).cpu().pin_memory()
    dw = torch.empty(out, cin, device=DEV)
    native.sf_checkpoint_wgrad(dy, native.checkpoint(hq, hs, 32), dw)
    native.sf_sync_status()
    ref, mag = oc.weight_grad(f64(dy.float()), oc.restore(f64(q.float()), f64(scale.float()), 32))
    close("dw", dw, ref, stored(F32, ref, _sum(tokens) * mag))


def test_no_tokens_give_the_base():
    dy, q = torch.empty(0, 64, dtype=BF, device=DEV), torch.empty(0, 48, dtype=E4, device=DEV)
    ck = native.checkpoint(q, torch.empty(0, 2, dtype=torch.uint8, device=DEV), 32)
    dw = torch.full((64, 48), 3.0, device=DEV)
    base = torch.randn(64, 48, device=DEV)
    native.sf_checkpoint_wgrad(dy, ck, dw, base=base)
    assert torch.equal(dw, base)
    native.sf_checkpoint_wgrad(dy, ck, dw)
    native.sf_sync_status()
    assert not dw.any()


def test_special_values_reach_their_entries_only():
    tokens, out, cin = 70, 264, 272
    dy = synth.normal((tokens, out), 1.0, 81).to(BF).to(DEV)
    x = synth.normal((tokens, cin), 1.0, 82).to(BF).to(DEV)
    x[3, 17] = float("nan")
    dy[5, 9] = float("inf")
    ck, _, _ = make_checkpoint(x, 32)
    dw = torch.empty(out, cin, device=DEV)
    ws = torch.empty(max(16, native.sf_checkpoint_wgrad_workspace_bytes(tokens, out, cin)), dtype=torch.uint8, device=DEV)
    native.sf_checkpoint_wgrad(dy, ck, dw, ws=ws)
    bad = ~torch.isfinite(dw)
    want = torch.zeros_like(bad)
    want[:, 17] = True
    want[9] = True
    assert torch.equal(bad, want)


def test_same_bits_on_a_side_stream_and_in_a_graph():
    tokens, out, cin = 700, 520, 528
    dy = synth.normal((tokens, out), 1.0, 91).to(BF).to(DEV)
    ck, _, _ = make_checkpoint(synth.normal((tokens, cin), 1.0, 92).to(BF).to(DEV), 128)
    ws = torch.empty(max(16, native.sf_checkpoint_wgrad_workspace_bytes(tokens, out, cin)), dtype=torch.uint8, device=DEV)
    dw = [torch.empty(out, cin, dtype=BF, device=DEV) for _ in range(3)]
    native.sf_checkpoint_wgrad(dy, ck, dw[0], ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        native.sf_checkpoint_wgrad(dy, ck, dw[1], ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        native.sf_checkpoint_wgrad(dy, ck, dw[2], ws=ws)
    g.replay()
    native.sf_sync_status()
    assert torch.equal(dw[0], dw[1]) and torch.equal(dw[0], dw[2])


def test_every_call_over_several_waves_gives_the_same_right_bits():
    # more tiles than pairs, split ones among them, a base that keeps the epilogues behind the products
    for tokens, out, cin, dt in ((2048, 4096, 4096, F32), (1030, 2600, 2048, F32), (640, 4352, 4352, BF)):
        dy = torch.empty(tokens, out, dtype=BF, device=DEV)
        x = torch.empty(tokens, cin, dtype=BF, device=DEV)
        base = torch.empty(out, cin, dtype=dt, device=DEV)
        for i, t in enumerate((dy, x, base)):
            synth.fill_normal_(t, 1.0, 101 + i)
        ck, q, scale = make_checkpoint(x, 64)
        native.sf_checkpoint_load(ck, x)          # exact in bf16
        ref = dy.double().t() @ x.double() + base.double()
        mag = dy.double().abs().t() @ x.double().abs() + base.double().abs()
        ws = torch.empty(max(16, native.sf_checkpoint_wgrad_workspace_bytes(tokens, out, cin)), dtype=torch.uint8, device=DEV)
        first = None
        for k in range(25):
            ws.fill_(255)
            dw = torch.full((out, cin), 7.0, dtype=dt, device=DEV)
            native.sf_checkpoint_wgrad(dy, ck, dw, base=base, ws=ws)
            if first is None:
                first = dw
                half = 2.0 ** -8 if dt == BF else 2.0 ** -24
                assert bool(((dw.double() - ref).abs() <= _sum(tokens) * mag + half * ref.abs()).all())
            assert torch.equal(dw, first), k
        native.sf_sync_status()


# as above, of the form that converts X on its way (few tokens, or outputs below 2048): a pair's second item and later ones
@pytest.mark.parametrize("tokens,out,cin,dt,group", [(256, 4096, 4096, F32, 64), (256, 4096, 4096, BF, 128), (448, 2600, 2048, F32, 32),
                                                     (500, 5000, 1200, BF, 0), (2048, 1024, 12288, F32, 64), (2100, 1900, 5008, BF, 32)])
def test_every_converted_call_over_several_waves_gives_the_same_right_bits(tokens, out, cin, dt, group):
    dy = torch.empty(tokens, out, dtype=BF, device=DEV)
    x = torch.empty(tokens, cin, dtype=BF, device=DEV)
    base = torch.empty(out, cin, dtype=dt, device=DEV)
    for i, t in enumerate((dy, x, base)):
        synth.fill_normal_(t, 1.0, 111 + i)
    ck, q, scale = make_checkpoint(x, group)
    native.sf_checkpoint_load(ck, x)          # exact in bf16
    ref = dy.double().t() @ x.double() + base.double()
    mag = dy.double().abs().t() @ x.double().abs() + base.double().abs()
    ws = torch.empty(max(16, native.sf_checkpoint_wgrad_workspace_bytes(tokens, out, cin)), dtype=torch.uint8, device=DEV)
    first = None
    for k in range(25):
        ws.fill_(255)
        dw = torch.full((out, cin), 7.0, dtype=dt, device=DEV)
        native.sf_checkpoint_wgrad(dy, ck, dw, base=base, ws=ws)
        if first is None:
            first = dw
            half = 2.0 ** -8 if dt == BF else 2.0 ** -24
            assert bool(((dw.double() - ref).abs() <= _sum(tokens) * mag + half * ref.abs()).all())
        assert torch.equal(dw, first), k
    native.sf_sync_status()


# converted on the way, restored first, on the CUDA cores; tokens that end inside a slab
@pytest.mark.parametrize("tokens,out,cin", [(130, 264, 256), (1, 40, 64), (521, 2048, 256), (130, 264, 250)])
def test_an_infinite_scale_of_the_last_token(tokens, out, cin):
    h8 = synth.normal((tokens, cin), 50.0, 121).abs().clamp(1, 448).to(DEV).to(E4)
    scale = torch.rand(tokens, -(-cin // 32), device=DEV) + 0.1
    scale[-1, 1] = float("inf")
    dy = synth.normal((tokens, out), 1.0, 122).abs().clamp(min=0.1).to(BF).to(DEV)
    dy[-1, ::3] *= -1
    dw = torch.empty(out, cin, device=DEV)
    ws = torch.empty(max(16, native.sf_checkpoint_wgrad_workspace_bytes(tokens, out, cin)), dtype=torch.uint8, device=DEV)
    native.sf_checkpoint_wgrad(dy, native.checkpoint(h8, scale, 32), dw, ws=ws)
    native.sf_sync_status()
    got = f64(dw)
    assert np.array_equal(got[:, 32:64], np.broadcast_to(np.sign(f64(dy[-1].float()))[:, None] * np.inf, (out, 32)))
    assert np.isfinite(got[:, :32]).all() and np.isfinite(got[:, 64:]).all()


def test_outputs_of_more_rows_than_a_grids_second_axis():
    # 64 rows a block: 2^16 blocks and more, without tokens, and with one whose rows no tensor copy takes
    out, cin = 64 * 65536 + 5, 3
    q, scale = torch.full((1, cin), 1.5, device=DEV).to(E4), torch.full((1, 1), 128, dtype=torch.uint8, device=DEV)
    base = torch.randn(out, cin, device=DEV)
    dw = torch.empty_like(base)
    native.sf_checkpoint_wgrad(torch.empty(0, out, dtype=BF, device=DEV), native.checkpoint(q[:0], scale[:0], 32), dw, base=base)
    native.sf_sync_status()
    assert torch.equal(dw, base)
    dy = torch.randn(1, out, device=DEV).to(BF)
    native.sf_checkpoint_wgrad(dy, native.checkpoint(q, scale, 32), dw)
    native.sf_sync_status()
    assert torch.equal(dw, (3.0 * dy.float()).t().expand(out, cin))


@pytest.mark.parametrize("tokens,out,cin", [(130, 264, 256), (521, 2048, 256), (130, 264, 250)])
def test_values_below_bf16s_least_normal_one(tokens, out, cin):
    # every code under scales of 2^-124: bf16's subnormal range, exact there, enters the products as it is
    codes = torch.arange(tokens * cin, dtype=torch.int64).remainder(127).to(torch.uint8)      # 0 .. 448, no NaN
    q = (codes | (torch.arange(tokens * cin) % 2 * 128).to(torch.uint8)).view(tokens, cin).to(DEV).view(E4)
    scale = torch.full((tokens, 1), 3, dtype=torch.uint8, device=DEV)
    scale[::2] = 5
    dy = synth.normal((tokens, out), 2.0 ** 30, 131).to(BF).to(DEV)
    dw = torch.empty(out, cin, device=DEV)
    ws = torch.empty(max(16, native.sf_checkpoint_wgrad_workspace_bytes(tokens, out, cin)), dtype=torch.uint8, device=DEV)
    native.sf_checkpoint_wgrad(dy, native.checkpoint(q, scale), dw, ws=ws)
    native.sf_sync_status()
    ref, mag = oc.weight_grad(f64(dy.float()), f64(q.float()) * np.exp2(f64(scale.float()) - 127.0))
    close("dw", dw, ref, stored(F32, ref, _sum(tokens) * mag))
