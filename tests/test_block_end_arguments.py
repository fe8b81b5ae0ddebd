"""Arguments of a residual block's end and its checkpoints that are settled on the host (CPU only).

Addresses are made up: every call here is refused, or has no rows and launches nothing.
"""

import pytest

from layer_optimizer_gb300 import build, native

BF, F32, E4, E8 = native.SF_BF16, native.SF_FP32, native.SF_E4M3, native.SF_E8M0
AT = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return native.load()


def _m(rows, cols, dtype, at=AT, ld=None):
    return native.sf_matrix(at, rows, cols, cols if ld is None else ld, dtype)


def _c(rows, cols, group=32, scale=AT, scale_dtype=E8, dtype=E4, at=AT):
    return native.sf_checkpoint(_m(rows, cols, dtype, at), scale, scale_dtype, group)


def _refused(match, call, status=native.SF_ERR_INVALID):
    with pytest.raises(native.SfError, match=match) as e:
        call()
    assert e.value.status == status


def test_checkpoint_arguments():
    x = _m(4, 64, BF)
    for call in (lambda c: native.sf_checkpoint_store(x, c), lambda c: native.sf_checkpoint_load(c, x)):
        _refused("checkpoint is NULL", lambda: call(None))
        _refused("checkpoint is 4 x 65", lambda: call(_c(4, 65)))
        _refused("type 0", lambda: call(_c(4, 64, dtype=BF)), native.SF_ERR_UNSUPPORTED)
        _refused("group must be", lambda: call(_c(4, 64, group=16)))
        _refused("group must be", lambda: call(_c(4, 64, group=-32)))
        _refused("scale is NULL", lambda: call(_c(4, 64, scale=None)))
        _refused("data is NULL", lambda: call(_c(4, 64, at=None)))
        _refused("scales of type 0", lambda: call(_c(4, 64, scale_dtype=BF)), native.SF_ERR_UNSUPPORTED)
    _refused("scales of type 1", lambda: native.sf_checkpoint_store(x, _c(4, 64, scale_dtype=F32)), native.SF_ERR_UNSUPPORTED)
    _refused("checkpoint is not aligned", lambda: native.sf_checkpoint_load(_c(4, 64, scale=AT + 2, scale_dtype=F32), x))
    _refused("x is NULL", lambda: native.sf_checkpoint_store(None, _c(4, 64)))
    _refused("y is NULL", lambda: native.sf_checkpoint_load(_c(4, 64), None))
    _refused("x: type 2", lambda: native.sf_checkpoint_store(_m(4, 64, E4), _c(4, 64)), native.SF_ERR_UNSUPPORTED)
    _refused("ld 63", lambda: native.sf_checkpoint_store(_m(4, 64, BF, ld=63), _c(4, 64)))
    load = lambda **kw: native.sf_checkpoint_load(_c(4, 64), x, **kw)  # noqa: E731
    _refused("row_factor is not aligned", lambda: load(row_factor=AT + 2))
    _refused("gain is not aligned", lambda: load(gain=AT + 2, gain_dtype=F32))
    _refused("gain: type 2", lambda: load(gain=AT, gain_dtype=E4), native.SF_ERR_UNSUPPORTED)
    _refused("gain_offset", lambda: load(gain=AT, gain_dtype=BF, gain_offset=float("nan")))
    _refused("gain_dtype", lambda: load(gain=AT))
    wide = 1 << 30
    _refused("2\\^30 columns", lambda: native.sf_checkpoint_store(_m(1, wide, BF), _c(1, wide)), native.SF_ERR_UNSUPPORTED)
    _refused("2\\^30 columns", lambda: native.sf_checkpoint_load(_c(1, wide), _m(1, wide, BF)), native.SF_ERR_UNSUPPORTED)
    # nothing to do
    native.sf_checkpoint_store(_m(0, 64, BF), _c(0, 64))
    native.sf_checkpoint_load(_c(0, 64, scale=None), _m(0, 64, F32))
    native.sf_checkpoint_load(_c(4, 0, group=0), _m(4, 0, F32))


def test_weight_gradient_arguments():
    dy, c, dw = _m(40, 64, BF), _c(40, 96), _m(64, 96, F32)
    ws = type("Workspace", (), dict(is_cuda=True, nbytes=1 << 40, is_contiguous=lambda s: True, data_ptr=lambda s: AT))()
    call = lambda dy=dy, c=c, dw=dw, **kw: native.sf_checkpoint_wgrad(dy, c, dw, ws=ws, **kw)  # noqa: E731
    _refused("dY is NULL", lambda: call(dy=None))
    _refused("dW is NULL", lambda: call(dw=None))
    _refused("checkpoint is NULL", lambda: call(c=None))
    _refused("dY: type 1", lambda: call(dy=_m(40, 64, F32)), native.SF_ERR_UNSUPPORTED)
    _refused("dW: type 2", lambda: call(dw=_m(64, 96, E4)), native.SF_ERR_UNSUPPORTED)
    _refused("dW is 63 x 96", lambda: call(dw=_m(63, 96, F32)))
    _refused("checkpoint is 40 x 96", lambda: call(dw=_m(64, 95, F32)))
    _refused("checkpoint is 41 x 96", lambda: call(c=_c(41, 96)))
    _refused("base: type 0", lambda: call(base=_m(64, 96, BF)), native.SF_ERR_UNSUPPORTED)
    _refused("base is 64 x 95", lambda: call(base=_m(64, 95, F32)))
    native.sf_checkpoint_wgrad(_m(40, 0, BF), _c(40, 96), _m(0, 96, F32), ws=ws)
    # every output reads all tokens of both operands
    _refused("must not lie over", lambda: native.sf_checkpoint_wgrad(_m(40, 40, BF, 2 * AT), _c(40, 40), _m(40, 40, BF, 2 * AT)))
    _refused("must not lie over", lambda: native.sf_checkpoint_wgrad(_m(40, 64, BF, 2 * AT), _c(40, 96), dw))
    # a workspace that is needed: too small, missing, or no memory of this device (an address that the driver does not know)
    dy, c, dw = _m(4096, 4096, BF), _c(4096, 4096), _m(4096, 4096, BF)
    need = native.sf_checkpoint_wgrad_workspace_bytes(4096, 4096, 4096)
    assert need > 2 * 4096 * 4096 and native.sf_checkpoint_wgrad_workspace_bytes(64, 4096, 4096) == 0
    _refused(f"workspace needs {need}", lambda: native.sf_checkpoint_wgrad(dy, c, dw))
    ws.nbytes = need
    _refused("ws must be device memory", lambda: native.sf_checkpoint_wgrad(dy, c, dw, ws=ws))


FULL = dict(residual=_m(8, 64, BF), gain_post=AT, gain_pre=AT, gain_dtype=F32, sum=_m(8, 64, BF), h=_m(8, 64, BF))


def _fwd(p=None, x=None, **kw):
    native.sf_sandwich_norm_forward(p if p is not None else native.sandwich(1e-5), x if x is not None else _m(8, 64, BF), **dict(FULL, **kw))


def test_forward_arguments():
    for name, bad in (("eps", -1.0), ("eps", float("inf")), ("residual_scale", float("nan")), ("block_scale", float("inf")),
                      ("gain_offset", float("nan")), ("gate_span", -1)):
        p = native.sandwich(**dict(dict(eps=1e-5), **{name: bad}))
        _refused(name, lambda: _fwd(p))
    _refused("configuration", lambda: native.sf_sandwich_norm_forward(None, _m(8, 64, BF), **FULL))
    _refused("x is NULL", lambda: native.sf_sandwich_norm_forward(native.sandwich(1e-5), None, **FULL))
    _refused("16384 columns", lambda: native.sf_sandwich_norm_forward(native.sandwich(1e-5), _m(8, 16385, BF), h=_m(8, 16385, BF), gain_pre=AT,
                                                                     gain_dtype=BF), native.SF_ERR_UNSUPPORTED)
    _refused("residual is 7 x 64", lambda: _fwd(residual=_m(7, 64, BF)))
    _refused("residual and sum", lambda: _fwd(sum=_m(8, 64, F32)))
    _refused("h: type 1", lambda: _fwd(h=_m(8, 64, F32)), native.SF_ERR_UNSUPPORTED)
    _refused("all NULL", lambda: _fwd(sum=None, h=None))
    _refused("gain_pre", lambda: _fwd(gain_pre=None))
    _refused("gain_pre", lambda: _fwd(gain_pre=None, h=None, rstd_pre=AT))
    _refused("rstd_post needs", lambda: _fwd(gain_post=None, rstd_post=AT))
    _refused("gain_post is not aligned", lambda: _fwd(gain_post=AT + 2))
    _refused("rstd_pre is not aligned", lambda: _fwd(rstd_pre=AT + 2))
    _refused("x8: scales", lambda: _fwd(x8=_c(8, 64, scale_dtype=F32)), native.SF_ERR_UNSUPPORTED)
    _refused("sum8 is 8 x 63", lambda: _fwd(sum8=_c(8, 63)))
    # a gate row for each span, the last one ragged
    p = native.sandwich(1e-5, gate_span=3)
    _refused("gate is 2 x 64, expected 3 x 64", lambda: _fwd(p, gate=_m(2, 64, F32)))
    _refused("gate is 8 x 64, expected 1 x 64", lambda: _fwd(gate=_m(8, 64, F32)))
    _refused("gate: type 2", lambda: _fwd(p, gate=_m(3, 64, E4)), native.SF_ERR_UNSUPPORTED)
    native.sf_sandwich_norm_forward(p, _m(0, 64, BF), gain_pre=AT, gain_dtype=F32, h=_m(0, 64, BF), gate=_m(0, 64, BF))


def _bwd(p=None, **kw):
    ws = type("Workspace", (), dict(is_cuda=True, nbytes=kw.pop("ws_bytes", 1 << 40), is_contiguous=lambda s: True,
                                    data_ptr=lambda s: AT))()
    args = dict(dh=_m(8, 64, BF), dsum=_m(8, 64, BF), x=_m(8, 64, BF), sum=_m(8, 64, BF), gain_post=AT, gain_pre=AT, gain_dtype=F32,
                rstd_post=AT, rstd_pre=AT, dresidual=_m(8, 64, BF), dx=_m(8, 64, BF), dgain_post=AT, dgain_pre=AT, dgain_dtype=F32, ws=ws)
    native.sf_sandwich_norm_backward(p if p is not None else native.sandwich(1e-5), **dict(args, **kw))


def test_backward_arguments():
    _refused("dh and dsum are NULL", lambda: _bwd(dh=None, dsum=None))
    _refused("no gradient", lambda: _bwd(dresidual=None, dx=None, dgain_post=None, dgain_pre=None))
    _refused("dh needs gain_pre", lambda: _bwd(gain_pre=None, dgain_pre=None))
    _refused("dh needs sum", lambda: _bwd(sum=None))
    _refused("dh needs rstd_pre", lambda: _bwd(rstd_pre=None))
    _refused("dgain_pre needs dh", lambda: _bwd(dh=None))
    _refused("dgain_post needs gain_post", lambda: _bwd(gain_post=None))
    _refused("dgate needs gate", lambda: _bwd(dgate=_m(1, 64, F32)))
    _refused("need x or x8", lambda: _bwd(x=None))
    _refused("needs rstd_post", lambda: _bwd(rstd_post=None))
    _refused("sum: type 1", lambda: _bwd(sum=_m(8, 64, F32)), native.SF_ERR_UNSUPPORTED)
    _refused("dx: type 1", lambda: _bwd(dx=_m(8, 64, F32)), native.SF_ERR_UNSUPPORTED)
    _refused("x is 9 x 64", lambda: _bwd(x=_m(9, 64, BF)))
    _refused("x8: group", lambda: _bwd(x=_c(8, 64, group=48)))
    _refused("sum8: scale is NULL", lambda: _bwd(sum=_c(8, 64, scale=None)))
    _refused("dgain_pre is not aligned", lambda: _bwd(dgain_pre=AT + 2))
    _refused("dgate is 2 x 64", lambda: _bwd(gate=_m(1, 64, F32), dgate=_m(2, 64, F32)))
    _refused("gate is 1 x 64, expected 4 x 64", lambda: _bwd(native.sandwich(1e-5, gate_span=2), gate=_m(1, 64, F32)))
    p = native.sandwich(1e-5, gate_span=1)
    for out in ("dresidual", "dx"):
        others = {"dresidual": _m(8, 64, BF, 2 * AT), "dx": _m(8, 64, BF, 2 * AT)}
        _refused("must not lie over the gate", lambda: _bwd(p, gate=_m(8, 64, BF), **dict(others, **{out: _m(8, 64, BF)})))
    need = native.sf_sandwich_norm_workspace_bytes(8, 64)
    _refused(f"workspace needs {need} bytes", lambda: _bwd(ws_bytes=need - 1))
    _refused("workspace needs", lambda: _bwd(ws=None))


def test_workspace_sizes():
    assert native.sf_sandwich_norm_workspace_bytes(-1, 64) == native.sf_sandwich_norm_workspace_bytes(8, 0) == 0
    assert native.sf_sandwich_norm_workspace_bytes(8, 16385) == 0
    assert native.sf_sandwich_norm_workspace_bytes(3, 64) == 2 * 3 * 64 * 4
    assert native.sf_sandwich_norm_workspace_bytes(10 ** 9, 16384) == 2 * 1024 * 16384 * 4
    assert native.sf_sandwich_norm_workspace_bytes(10 ** 9, 64) == 2 * 8192 * 64 * 4


# a gradient of `rows` rows by a gate of 16 x 96 whose rows lie `step` bytes apart: (rows, bytes behind the gate, distance of rows, meet)
def _places(size, step):
    width, last = 96 * size, 15 * step
    return [(64, 0, step, True), (64, step, step, True), (64, -step, step, True), (64, size, step, True), (64, size - width, step, True),
            (64, width, step, False), (64, -width, step, False), (64, width - size, step, True),                          # side by side, and one column less
            (64, last + width, step, False), (64, last + width - size, step, True), (64, last, step, True), (64, last + step, step, False),
            (64, -63 * step - width, step, False), (64, -63 * step - width + size, step, True), (64, -64 * step, step, False),
            (16, 5 * step + width, step, False), (16, 5 * step - size, step, True), (16, width, step + size, True)]      # another distance: by the ends


@pytest.mark.parametrize("dt,size", [(F32, 4), (BF, 2)])
@pytest.mark.parametrize("name", ["dresidual", "dx", "dgate"])
def test_overlaps_are_told_by_their_elements(dt, size, name):
    """A gradient that does not meet the gate goes on to the refusal of a workspace that is too small."""
    at, ld = 64 * AT, 400
    for rows, off, step, meet in _places(size, ld * size):
        n = 16 if name == "dgate" else rows
        if n != rows:
            continue
        total = 64 if name == "dgate" else rows
        p = native.sandwich(1e-5, gate_span=-(-total // 16))
        far = {k: _m(total, 96, dt, a * AT) for k, a in (("dh", 1), ("dsum", 2), ("x", 4), ("sum", 8), ("dresidual", 16), ("dx", 32))}
        out = native.sf_matrix(at + off, n, 96, step // size, dt)
        _refused("the gate" if meet else "workspace needs",
                 lambda: _bwd(p, gate=native.sf_matrix(at, 16, 96, ld, dt), **dict(far, **{name: out}), ws_bytes=0))  # noqa: B023
    # a gate of one row, between the rows of a wider buffer and on them
    far = {k: _m(64, 96, dt, a * AT) for k, a in (("dh", 1), ("dsum", 2), ("x", 4), ("sum", 8), ("dresidual", 16), ("dx", 32))}
    if name != "dgate":
        for off, meet in ((7 * ld + 96, False), (7 * ld + 95, True), (7 * ld - 96, False), (7 * ld - 95, True), (-96, False), (63 * ld + 96, False)):
            far[name] = native.sf_matrix(at, 64, 96, ld, dt)
            _refused("the gate" if meet else "workspace needs",
                     lambda: _bwd(gate=native.sf_matrix(at + off * size, 1, 96, 0, dt), **far, ws_bytes=0))  # noqa: B023


def test_weight_gradients_over_a_part_of_an_operand():
    at = 4 * AT
    dw = native.sf_matrix(at, 64, 96, 400, BF)
    away = dict(at=32 * AT, scale=64 * AT)
    dy, c = _m(40, 64, BF, at=128 * AT), _c(40, 96, **away)
    for d in (_m(40, 64, BF, at=at + 2), _m(40, 64, BF, at=at - 2), native.sf_matrix(at + 800, 40, 64, 400, BF), native.sf_matrix(at - 126, 40, 64, 400, BF)):
        _refused("must not lie over", lambda: native.sf_checkpoint_wgrad(d, c, dw))
    _refused("must not lie over", lambda: native.sf_checkpoint_wgrad(dy, _c(40, 96, at=at + 100, scale=64 * AT), dw))
    for scale in (at, at + 190, at + 800 * 63 + 191, at - 40 * 3 + 1):
        _refused("must not lie over", lambda: native.sf_checkpoint_wgrad(dy, _c(40, 96, at=32 * AT, scale=scale), dw))
    for base in (native.sf_matrix(at, 64, 96, 401, BF), native.sf_matrix(at + 800, 64, 96, 400, BF), native.sf_matrix(at - 2, 64, 96, 400, BF)):
        _refused("dW lies over base", lambda: native.sf_checkpoint_wgrad(dy, c, dw, base=base))


def test_outputs_over_a_part_of_the_gate():
    at = 4 * AT
    p, each = native.sandwich(1e-5, gate_span=4), native.sandwich(1e-5, gate_span=1)
    far = dict(residual=_m(8, 64, BF, 16 * AT), sum=_m(8, 64, BF, 32 * AT), h=_m(8, 64, BF, 64 * AT))
    for out in ("sum", "h"):
        for place in (at, at + 128, at - 8 * 128 + 2, at + 2 * 128 - 2):          # over a gate of 2 rows
            _refused("over the gate", lambda: _fwd(p, gate=_m(2, 64, BF, at), **dict(far, **{out: _m(8, 64, BF, place)})))
        for gate in (_m(8, 64, BF, at + 128), _m(8, 64, F32, at), _m(8, 64, BF, at, ld=65), _m(8, 64, BF, at + 2)):
            _refused("over the gate", lambda: _fwd(each, gate=gate, **dict(far, **{out: _m(8, 64, BF, at)})))
    outs = dict(dresidual=_m(8, 64, BF, 16 * AT), dx=_m(8, 64, BF, 32 * AT))
    for out in outs:
        for place in (at + 2, at + 128, at - 8 * 128 + 2, at + 2 * 128 - 2):
            _refused("must not lie over the gate", lambda: _bwd(p, gate=_m(2, 64, BF, at), **dict(outs, **{out: _m(8, 64, BF, place)})))
    for dgate in (_m(2, 64, F32, at), _m(2, 64, BF, at, ld=65), _m(2, 64, BF, at + 128), _m(2, 64, BF, at + 2), _m(2, 64, BF, at - 2 * 128 + 2)):
        _refused("dgate lies over the gate", lambda: _bwd(p, gate=_m(2, 64, BF, at), dgate=dgate, **outs))
    _refused("dgate lies over the gate", lambda: _bwd(gate=_m(1, 64, BF, at), dgate=_m(1, 64, F32, at), **outs))
