"""GPU: a linear layer's gradients one at a time, from no more than each reads."""
import pytest
import torch

import block_scaled_fp4_e2m1_amd as bs
from test_gpu_fp8 import DEV, gen, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(0, 32, 48), (1, 16, 16), (130, 256, 528), (777, 1552, 2064)])
def test_one_gradient(M, N, K):
    g = gen(M + N + K)
    x, dy, W = rows(g, M, K), rows(g, M, N, 1e-2), rows(g, N, K, 0.02)
    _, _, WT, SWT = bs.fp8_quantize_weight(W, transposed=True)
    for dtype in (torch.bfloat16, torch.float32):
        dx, none = bs.fp8_linear_backward(dy, None, WT, SWT, need_dW=False, dW_dtype=dtype)
        assert none is None and torch.equal(dx, bs.fp8_linear_backward(dy, x, WT, SWT, need_dW=False)[0])
        none, dW = bs.fp8_linear_backward(dy, x, None, None, need_dx=False, dW_dtype=dtype)
        assert none is None and torch.equal(dW, bs.fp8_linear_backward(dy, x, WT, SWT, need_dx=False, dW_dtype=dtype)[1])
    assert bs.fp8_linear_backward(dy, None, None, None, need_dx=False, need_dW=False) == (None, None)
