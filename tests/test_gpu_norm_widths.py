"""The staged norm backward at widths whose blocks have 96 threads (GPU).

Rows of 257 to 384 units of eight columns take blocks of 96 threads, one row each; bounds and
checks are those of test_gpu_norm.py.
"""

import pytest
import torch

import test_gpu_norm as base

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("rows,cols,pad", [(400, 2560, 0), (330, 2056, 8), (700, 3064, 0), (350, 2561, 0), (330, 3059, 2)])
@pytest.mark.parametrize("at,st,p", [(BF, BF, 0.1), (F32, F32, 0.0), (BF, F32, 0.25)])
def test_blocks_of_96_threads(rows, cols, pad, at, st, p):
    base.test_add_rmsnorm_backward_matches_oracle(rows, cols, pad, 0, at, st, BF, F32, True, p)
