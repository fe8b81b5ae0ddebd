"""8-bit checkpoints, written and read, against the fp64 oracle (GPU).

Writing is exact arithmetic (a scale by comparison, a product with a power of two, one rounding), so scales and values
must be the oracle's.  Reading: the product with a power of two is exact, then at most a factor, a gain with its offset
(added in fp32) and their products: four roundings of 2^-24; then the output type's rounding.
"""

import numpy as np
import pytest
import torch

from _block_end import BF, DEV, E4, E8, F32, SHAPES, U, close, guard_ok, make_checkpoint, new_checkpoint, rows_of, stored
from _util import f64
from layer_optimizer_gb300 import native, synth
from oracle import checkpoint as oc

pytestmark = pytest.mark.gpu
LONG = [(3, 16400, 0, 0), (2, 40001, 0, 0), (2, 40000, 0, 0), (400, 20000, 0, 0)]      # longer than a thread's registers hold


def _same(q, scale, v, group):
    rq, rs = oc.quantize(v, group)
    assert np.array_equal(f64(scale.float()).reshape(rs.shape), rs)
    assert np.array_equal(f64(q.float()), rq, equal_nan=True)


@pytest.mark.parametrize("rows,cols,pad,lead", SHAPES + LONG)
@pytest.mark.parametrize("xt,group", [(BF, 32), (BF, 128), (F32, 64), (F32, 0), (BF, 0)])
def test_store_is_the_oracles(rows, cols, pad, lead, xt, group):
    x, _ = rows_of(rows, cols, pad, xt, 1 + rows + cols, 3.0, lead)
    ck, q, scale, buf = new_checkpoint(rows, cols, group, pad, lead)
    native.sf_checkpoint_store(x, ck)
    native.sf_sync_status()
    _same(q, scale, f64(x.float()), group)
    assert guard_ok(q, buf, lead)


@pytest.mark.parametrize("cols", [96, 100, 75, 512, 603, 1037])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_next_to_the_largest_value(cols, group, xt, bad):
    # in every place around it: its scale and its group's other values are those of the finite ones
    x = synth.normal((64, cols), 1.0, 4).to(xt).to(DEV)
    for i in range(64):
        x[i, i] = 300.0
        x[i, (i + i % 7 + 1) % cols] = bad
        x[i, (i + 64) % cols if i % 2 else (i + 33) % cols] = -bad
    ck, q, scale, _ = new_checkpoint(64, cols, group)
    native.sf_checkpoint_store(x, ck)
    _same(q, scale, f64(x.float()), group)


@pytest.mark.parametrize("cols", [96, 75, 603, 1037])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("xt", [BF, F32])
def test_store_special_values(cols, group, xt):
    x = synth.normal((9, cols), 1.0, 3).to(xt).to(DEV)
    x[0] = 0.0
    x[1, 33], x[1, 2] = float("nan"), float("-inf")
    x[2] = float("inf")
    x[3] *= 2.0 ** -126                              # subnormal entries
    x[4] = 448.0 * 2.0 ** 5                          # the largest value exactly
    x[5] = torch.tensor(448.0 * 2.0 ** 5 * (1 + 2.0 ** -7), dtype=F32).to(xt)     # just above it: the next scale
    x[6, 0] = torch.finfo(xt).max
    x[7] = 2.0 ** -133                               # bf16's smallest
    x[8, :40] = -0.0
    ck, q, scale, _ = new_checkpoint(9, cols, group)
    native.sf_checkpoint_store(x, ck)
    _same(q, scale, f64(x.float()), group)


def _read(q, scale, group, cols):
    return oc.restore(f64(q.float()), f64(scale.float()).reshape(q.shape[0], -1), group)


@pytest.mark.parametrize("rows,cols,pad,lead", SHAPES + LONG)
@pytest.mark.parametrize("yt,group,factor,gt,offset", [
    (BF, 32, False, None, 0.0), (F32, 128, False, None, 0.0), (BF, 0, True, BF, 0.0), (F32, 64, True, F32, 1.0), (BF, 128, False, F32, 0.0),
])
def test_load_matches_oracle(rows, cols, pad, lead, yt, group, factor, gt, offset):
    x, _ = rows_of(rows, cols, pad, F32, 5 + rows + cols, 2.0, lead)
    ck, q, scale = make_checkpoint(x, group, pad, lead)
    y, buf = rows_of(rows, cols, pad, yt, None, lead=lead)
    f = torch.rand(rows, device=DEV) + 0.5 if factor else None
    gain = (1.0 - offset + synth.normal((cols,), 0.2, 6)).to(gt).to(DEV) if gt else None
    native.sf_checkpoint_load(ck, y, row_factor=f, gain=gain, gain_offset=offset)
    native.sf_sync_status()
    ref = _read(q, scale, group, cols)
    if factor:
        ref = ref * f64(f)[:, None]
    g_err = 0.0
    if gt:
        g = f64(gain.float())
        g_err = np.abs(ref) * U * np.abs(offset + g)
        ref = ref * (offset + g)
    err = 4 * U * np.abs(ref) + g_err if factor or gt else 0.0 * ref
    close("y", y, ref, stored(yt, ref, err) if yt == BF or factor or gt else err)
    if yt == F32 and not factor and not gt:
        assert np.array_equal(f64(y), ref)
    assert guard_ok(y, buf, lead)


@pytest.mark.parametrize("group", [0, 32, 128])
def test_load_of_the_norms_8_bit_output(group):
    rows, cols = 65, 1000
    x = synth.normal((rows, cols), 1.0, 8).to(BF).to(DEV)
    gain = torch.ones(cols, dtype=BF, device=DEV)
    h, h8 = torch.empty_like(x), torch.empty(rows, cols, dtype=E4, device=DEV)
    scale = torch.empty(rows, -(-cols // group) if group else 1, device=DEV)
    native.sf_add_rmsnorm_forward(x, None, gain, 1e-5, h=h, h8=h8, h8_scale=scale, group=group)
    y = torch.empty(rows, cols, device=DEV)
    native.sf_checkpoint_load(native.checkpoint(h8, scale, group), y)
    ref = _read(h8, scale, group, cols)
    close("y", y, ref, U * np.abs(ref))
    # and it is h, within half a step of e4m3 (2^-4 relative, 2^-10 scales near zero) and h's own rounding to bf16
    s = oc.spread(f64(scale), group, cols)
    h = f64(h.float())
    assert np.all(np.abs(f64(y) - h) <= (2.0 ** -4 + 2.0 ** -8 + 1e-6) * np.abs(h) + 2.0 ** -10 * s)


def test_scales_of_every_code():
    # values 1.5 and a NaN under each code, read in fp32: 255 is NaN, 0 is 2^-127
    q = torch.full((256, 8), 1.5, device=DEV).to(E4)
    q[:, 7] = float("nan")
    codes = torch.arange(256, dtype=torch.uint8, device=DEV)
    y = torch.empty(256, 8, device=DEV)
    native.sf_checkpoint_load(native.checkpoint(q, codes), y)
    want = 1.5 * np.ldexp(1.0, np.arange(256) - 127)
    want[255] = np.nan
    got = f64(y)
    assert np.array_equal(got[:, 0], want, equal_nan=True) and np.isnan(got[:, 7]).all()


def test_no_rows_and_pinned_host_memory():
    ck, q, scale, _ = new_checkpoint(0, 64, 32)
    native.sf_checkpoint_store(torch.empty(0, 64, dtype=BF, device=DEV), ck)
    native.sf_checkpoint_load(ck, torch.empty(0, 64, dtype=BF, device=DEV))
    x = synth.normal((130, 640), 1.0, 9).to(BF).to(DEV)
    want, wq, ws = make_checkpoint(x, 64)
    hq, hs = torch.empty(130, 640, dtype=E4).pin_memory(), torch.empty(130, 10, dtype=E8).pin_memory()
    host = native.checkpoint(hq, hs, 64)
    native.sf_checkpoint_store(x, host)            # straight into host memory, and back
    y, w = torch.empty_like(x), torch.empty_like(x)
    native.sf_checkpoint_load(host, y)
    native.sf_checkpoint_load(want, w)
    native.sf_sync_status()
    assert torch.equal(hq.float(), wq.float().cpu()) and torch.equal(hs.view(torch.uint8), ws.view(torch.uint8).cpu())
    assert torch.equal(y, w)


def test_past_2_31_elements():
    rows, cols = 530001, 4096
    x = torch.empty(rows, cols, dtype=BF, device=DEV)
    synth.fill_normal_(x, 1.0, 5)
    ck, q, scale = make_checkpoint(x, 128)
    pick = [0, 1, 262144, 524287, 524288, 524289, rows - 1]
    _same(q[pick], scale.view(torch.uint8)[pick].view(E8), f64(x[pick].float()), 128)
    native.sf_checkpoint_load(ck, x)
    native.sf_sync_status()
    for i in pick:
        r = slice(i, i + 1)
        assert np.array_equal(f64(x[r].float()), _read(q[r], scale[r], 128, cols))


def test_streams_and_graphs():
    rows, cols = 200, 512
    x = synth.normal((rows, cols), 1.0, 10).to(BF).to(DEV)
    want, wq, ws = make_checkpoint(x, 32)
    ck, q, scale, _ = new_checkpoint(rows, cols, 32)
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        native.sf_checkpoint_store(x, ck)
        native.sf_checkpoint_load(ck, y)
    side.synchronize()
    assert torch.equal(q.float(), wq.float()) and torch.equal(scale.view(torch.uint8), ws.view(torch.uint8))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        native.sf_checkpoint_store(x, ck)
        native.sf_checkpoint_load(ck, y)
    x.copy_(synth.normal((rows, cols), 2.0, 11).to(BF))
    g.replay()
    torch.cuda.synchronize()
    _same(q, scale, f64(x.float()), 32)
    assert np.array_equal(f64(y.float()), _read(q, scale, 32, cols))


@pytest.mark.parametrize("cols", [96, 75, 104, 264, 520, 1037, 4096])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("xt", [BF, F32])
def test_groups_without_a_finite_value(cols, group, xt):
    # next to others, in every place: their scale is 2^-126
    x = synth.normal((40, cols), 1.0, 6).to(xt).to(DEV)
    x[1], x[2], x[3, ::2], x[3, 1::2] = float("nan"), float("inf"), float("nan"), float("-inf")
    for i in range(4, 40):
        c = 8 * i % cols
        x[i, c:c + 32 + 8 * (i % 13)] = float("nan") if i % 3 else float("inf")
        x[i, : i % 9 * 8] = float("nan")
    ck, q, scale, _ = new_checkpoint(40, cols, group)
    native.sf_checkpoint_store(x, ck)
    native.sf_sync_status()
    _same(q, scale, f64(x.float()), group)


@pytest.mark.parametrize("rows,cols,pad", [(64, 96, 0), (64, 75, 0), (64, 512, 0), (64, 603, 0), (64, 1037, 0), (400, 4096, 0), (64, 520, 8), (40, 20000, 0)])
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("xt", [BF, F32])
def test_the_sign_of_zero(rows, cols, pad, group, xt):
    # v / 2^k keeps it, and so does the rounding of what is far below e4m3's least value, whatever lies beside it
    x, _ = rows_of(rows, cols, pad, xt, 12 + cols, 1.0)
    x[:, 1::3] = -0.0
    x[:, 2::9] = 0.0
    x[:, 5::9] = -2.0 ** -30
    x[8::4, 7], x[9::4, 40] = float("inf"), float("nan")
    x[5] = -0.0
    ck, q, scale, _ = new_checkpoint(rows, cols, group, pad)
    native.sf_checkpoint_store(x, ck)
    native.sf_sync_status()
    _same(q, scale, f64(x.float()), group)
    codes, fine = q.view(torch.uint8), torch.isfinite(x)
    assert torch.equal((codes >> 7)[fine].bool(), torch.signbit(x)[fine])
    assert bool(((codes & 0x7f) == 0x7f)[~fine].all())


@pytest.mark.parametrize("cols,pad", [(256, 0), (264, 0), (253, 0), (603, 0)])
@pytest.mark.parametrize("yt", [BF, F32])
def test_every_value_under_the_smallest_scales(cols, pad, yt):
    # e4m3's quantum is 2^-9: exact in fp32 (to 2^-149) always, in bf16 (to 2^-133) from scales of 2^-124 on, else to its nearest
    codes = torch.arange(cols, dtype=torch.int32).remainder(256).to(torch.uint8).repeat(8, 1).to(DEV)
    q = torch.empty(8, cols + pad, dtype=E4, device=DEV)[:, :cols]
    q.copy_(codes.view(E4))
    scale = torch.tensor([0, 1, 2, 3, 4, 5, 120, 200], dtype=torch.uint8, device=DEV)
    y = torch.empty(8, cols, dtype=yt, device=DEV)
    native.sf_checkpoint_load(native.checkpoint(q, scale), y)
    native.sf_sync_status()
    ref = f64(q.float()) * np.ldexp(1.0, np.array([0, 1, 2, 3, 4, 5, 120, 200]) - 127)[:, None]
    got = f64(y.float())
    fine = np.isfinite(ref)
    assert np.isnan(got[~fine]).all()
    assert np.array_equal(got[fine], f64(torch.from_numpy(ref).to(yt).float())[fine])
    if yt == F32:
        assert np.array_equal(got[fine], ref[fine])
    else:
        assert np.array_equal(got[3:][fine[3:]], ref[3:][fine[3:]])
