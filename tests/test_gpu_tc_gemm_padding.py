"""The tensor-core GEMM leaves what lies between C's rows alone (GPU).

C may be a view of a wider buffer (ldc > N).  Whatever N is, the product's
stores stay inside its N columns and M rows, also where a 16-byte unit of a
row is only partly C's.  Values: within 1e-5 of sum |a||b|, the library's bound
for its GEMM.
"""

import numpy as np
import pytest
import torch

from _util import f64
from layer_optimizer_gb300 import native, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("M,N,K,ldc", [(64, 61, 64, 64), (300, 259, 72, 264), (33, 2, 8, 4), (130, 300, 128, 304), (40, 61, 64, 61)])
def test_padding_of_c_is_untouched(M, N, K, ldc, accumulate):
    A, B = synth.normal((M, K), 1.0, 1, dtype=torch.bfloat16), synth.normal((N, K), 1.0, 2, dtype=torch.bfloat16)
    buf = torch.full((M + 1, ldc), 7.0, device=DEV)
    native.sf_gemm_abt_bf16(A.to(DEV), B.to(DEV), buf, M, N, K, K, K, ldc, 1.0, accumulate)
    native.sf_sync_status()
    assert bool((buf[:M, N:] == 7.0).all()) and bool((buf[M:] == 7.0).all())
    a, b = f64(A.float()), f64(B.float())
    want = a @ b.T + (7.0 if accumulate else 0.0)
    assert np.all(np.abs(f64(buf[:M, :N]) - want) <= 1e-5 * (np.abs(a) @ np.abs(b).T + 7.0))
