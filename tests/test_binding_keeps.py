"""Structures made from tensors keep them alive as long as they live (CPU only: stand-ins for device tensors)."""

import gc
import weakref

import pytest
import torch

from layer_optimizer_gb300 import native


class _Tensor:
    """What the binding asks of a device tensor."""
    is_cuda = True
    data_ptr = lambda self: 1 << 20  # noqa: E731

    def __init__(self, shape, dtype):
        self.shape, self.dtype = shape, dtype

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (self.shape[-1], 1)

    def numel(self):
        return self.shape[0]

    def is_contiguous(self):
        return True


@pytest.fixture(autouse=True, scope="module")
def types():
    native._DTYPES[torch.bfloat16] = native.SF_BF16


def _alive(make, shape, dtype):
    """Whether the tensor lives as long as what is made from it, and no longer."""
    tensor = _Tensor(shape, dtype)
    ref = weakref.ref(tensor)
    made = make(tensor)
    del tensor
    gc.collect()
    alive = ref() is not None
    del made
    gc.collect()
    return alive, ref() is None


def test_a_generator_keeps_its_device_offset():
    # the kernel reads it when it runs, and again whenever a captured graph is replayed
    assert _alive(lambda t: native.rng(1, 0, t), (1,), torch.int64) == (True, True)


def test_a_matrix_keeps_its_tensor():
    assert _alive(native.matrix, (4, 8), torch.bfloat16) == (True, True)
    m = native.matrix(_Tensor((4, 8), torch.bfloat16))
    assert native.matrix(m) is m and (m.rows, m.cols, m.ld) == (4, 8, 8)
