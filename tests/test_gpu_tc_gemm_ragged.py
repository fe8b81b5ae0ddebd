"""The tensor-core GEMM with rows of C that end inside a 16-byte unit (GPU).

Whole boxes of 32 columns leave by tensor stores, the last columns element by
element: values (1e-5 of sum |a||b|, the library's bound for its GEMM) and the
padding, over several tiles, both operand layouts and accumulation.
"""

import numpy as np
import pytest
import torch

from _util import f64
from layer_optimizer_gb300 import native, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("M,N,K,ldc", [(300, 1023, 136, 1024), (513, 289, 64, 292), (40, 255, 200, 256), (257, 257, 72, 260), (600, 31, 64, 32),
                                       (70, 33, 64, 40), (128, 1, 64, 4)])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("mn", [False, True])
def test_ragged_rows(M, N, K, ldc, accumulate, mn):
    A, B = synth.normal((M, K), 1.0, 1, dtype=torch.bfloat16), synth.normal((N, K), 1.0, 2, dtype=torch.bfloat16)
    buf = torch.full((M + 1, ldc), 7.0, device=DEV)
    if mn:      # both operands stored transposed, rows padded to 16 bytes
        lda, ldb = M + -M % 8, N + -N % 8
        a, b = torch.zeros(K, lda, dtype=torch.bfloat16, device=DEV), torch.zeros(K, ldb, dtype=torch.bfloat16, device=DEV)
        a[:, :M], b[:, :N] = A.t().to(DEV), B.t().to(DEV)
        native.sf_gemm_bf16(a, 1, b, 1, buf, M, N, K, lda, ldb, ldc, 0.5, accumulate)
    else:
        native.sf_gemm_bf16(A.to(DEV), 0, B.to(DEV), 0, buf, M, N, K, K, K, ldc, 0.5, accumulate)
    native.sf_sync_status()
    assert bool((buf[:M, N:] == 7.0).all()) and bool((buf[M:] == 7.0).all())
    a, b = f64(A.float()), f64(B.float())
    want = 0.5 * (a @ b.T) + (7.0 if accumulate else 0.0)
    assert np.all(np.abs(f64(buf[:M, :N]) - want) <= 1e-5 * (np.abs(a) @ np.abs(b).T + 7.0))
