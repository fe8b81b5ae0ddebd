"""Arguments of the output end's operators that are settled on the host (CPU only)."""

import pytest

from layer_optimizer_gb300 import build, native


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return native.load()


@pytest.mark.parametrize("piece", [1024, 1 << 20, 1 << 40, 2 ** 63 - 1024, 2 ** 63 - 512, 2 ** 63 - 256])
@pytest.mark.parametrize("n,d,v", [(100, 64, 1000), (17, 61, 1), (300, 256, 1023)])
def test_a_piece_beyond_the_vocabulary_is_the_whole_of_it(n, d, v, piece):
    # every size of at least V is one piece, up to the type's largest multiple of 256
    assert native.lce_vocab_workspace_bytes(n, d, v, piece) == native.lce_vocab_workspace_bytes(n, d, v, 1024)


def _matrix(rows, cols, dtype, at=1 << 20):
    return native.sf_matrix(at, rows, cols, cols, dtype)


def test_vectors_given_by_address():
    # no rows: every check runs and nothing is launched
    x, s = _matrix(0, 64, native.SF_BF16), _matrix(0, 64, native.SF_FP32)
    native.sf_add_rmsnorm_forward(x, s, 4096, 1e-5, h=x, rstd=4096, gain_dtype=native.SF_BF16)
    native.sf_add_rmsnorm_backward(x, s, 4096, 4096, dx=x, gain_dtype=native.SF_FP32)
    with pytest.raises(native.SfError, match="gain_dtype"):
        native.sf_add_rmsnorm_forward(x, s, 4096, 1e-5, h=x)
    with pytest.raises(native.SfError, match="dgain_dtype"):
        native.sf_add_rmsnorm_backward(x, s, 4096, 4096, dx=x, gain_dtype=native.SF_BF16, dgain=4096)
    # a bf16 gain may lie on 2 bytes, an fp32 one may not
    native.sf_add_rmsnorm_forward(x, s, 4098, 1e-5, h=x, gain_dtype=native.SF_BF16)
    with pytest.raises(native.SfError, match="gain is not aligned"):
        native.sf_add_rmsnorm_forward(x, s, 4098, 1e-5, h=x, gain_dtype=native.SF_FP32)


def test_missing_arguments_are_the_librarys_errors():
    x = _matrix(0, 64, native.SF_BF16)
    for call in (lambda: native.sf_dropout(None, x, 0.0), lambda: native.sf_dropout(x, None, 0.0),
                 lambda: native.sf_add_rmsnorm_forward(None, None, 4096, 1e-5, h=x, gain_dtype=native.SF_BF16),
                 lambda: native.sf_add_rmsnorm_forward(x, None, None, 1e-5, h=x),
                 lambda: native.sf_add_rmsnorm_backward(None, x, 4096, 4096, dx=x, gain_dtype=native.SF_BF16),
                 lambda: native.sf_add_rmsnorm_backward(x, None, 4096, 4096, dx=x, gain_dtype=native.SF_BF16),
                 lambda: native.sf_add_rmsnorm_backward(x, x, None, 4096, dx=x),
                 lambda: native.lce_vocab_forward_backward(None, x, 4096), lambda: native.lce_vocab_forward_backward(x, None, 4096)):
        with pytest.raises(native.SfError, match="is NULL"):
            call()


def test_vectors_off_their_type_are_refused():
    # addresses that a kernel would fault on; no rows where the call would otherwise launch
    x = _matrix(0, 64, native.SF_BF16)
    q = _matrix(0, 64, native.SF_E4M3)
    bf = dict(gain_dtype=native.SF_BF16)
    odd = native.rng(1, 0, 4100)
    calls = {
        "rstd": [lambda: native.sf_add_rmsnorm_forward(x, None, 4096, 1e-5, h=x, rstd=4098, **bf),
                 lambda: native.sf_add_rmsnorm_backward(x, x, 4096, 4098, dx=x, **bf)],
        "h8_scale": [lambda: native.sf_add_rmsnorm_forward(x, None, 4096, 1e-5, h8=q, h8_scale=4098, **bf)],
        "device_offset": [lambda: native.sf_dropout(x, x, 0.5, odd),
                          lambda: native.sf_add_rmsnorm_forward(x, None, 4096, 1e-5, h=x, p=0.5, rng=odd, **bf),
                          lambda: native.sf_add_rmsnorm_backward(x, x, 4096, 4096, dx=x, p=0.5, rng=odd, **bf)],
    }
    H, W = _matrix(20, 64, native.SF_BF16), _matrix(300, 64, native.SF_BF16)
    for name in ("labels", "loss", "token_loss"):
        kw = {"labels": 4096, name: 4098}
        calls[name] = [lambda kw=kw: native.lce_vocab_forward_backward(H, W, **kw)]
    for name, each in calls.items():
        for call in each:
            with pytest.raises(native.SfError, match=f"{name} is not aligned"):
                call()


class _Pageable:
    """A workspace tensor in ordinary host memory."""
    is_cuda = False

    def is_pinned(self):
        return False

    def is_contiguous(self):
        return True

    nbytes = 1 << 20

    def data_ptr(self):
        return 1 << 21


class _Strided(_Pageable):
    is_cuda = True

    def is_contiguous(self):
        return False


@pytest.mark.parametrize("ws,match", [(_Pageable(), "device or pinned"), (_Strided(), "dense")])
def test_workspaces_that_the_device_cannot_use_are_refused(ws, match):
    x = _matrix(0, 64, native.SF_BF16)
    with pytest.raises(native.SfError, match=f"ws must be .*{match}"):
        native.sf_add_rmsnorm_backward(x, x, 4096, 4096, dx=x, ws=ws, gain_dtype=native.SF_BF16)
    with pytest.raises(native.SfError, match=f"ws must be .*{match}"):
        native.lce_vocab_forward_backward(_matrix(20, 64, native.SF_BF16), _matrix(300, 64, native.SF_BF16), 4096, ws=ws)
