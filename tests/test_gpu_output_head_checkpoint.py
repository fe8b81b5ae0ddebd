"""The example's 8-bit copy of h, read back (GPU)."""

import os
import sys

import pytest
import torch

from layer_optimizer_gb300 import native, synth

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import output_head  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hidden", [256, 1000])
def test_the_copy_restores_h(hidden):
    N, V = 48, 600
    x, r = (synth.normal((N, hidden), s, 5 + int(s), dtype=torch.bfloat16).cuda() for s in (1.0, 2.0))
    y = torch.arange(N, dtype=torch.int32, device="cuda")
    head = output_head.OutputHead(N, hidden, V, seed=5, checkpoint=True)
    head.forward_backward(x, r, y, 1)
    native.sf_sync_status()
    got, h = head.restored(), head.h.float()
    # half a quantum of e4m3 (4 significant bits: 2^-4 of the value; 2^-10 where it is subnormal) and of h's own bf16
    scale = head.h8_scale.repeat_interleave(128, dim=1)[:, :hidden]
    assert got.shape == h.shape
    assert bool(((got - h).abs() <= (2.0 ** -4 + 2.0 ** -7) * h.abs() + 2.0 ** -10 * scale).all())
