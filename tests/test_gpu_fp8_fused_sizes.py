"""GPU: the quantiser inside the E4M3 product gives the bits of the two calls at every size where it is taken."""
import pytest
import torch

import block_scaled_fp4_e2m1_amd as bs
import fp8_ref as R
from test_gpu_fp8 import DEV, codes, gen, rows, scales

pytestmark = pytest.mark.gpu


# one row of short sums and many columns, on either side of 8192 and 16384 columns and of K K / 128
@pytest.mark.parametrize("M,N,K", [(1, 8192, 512), (1, 8200, 512), (1, 16384, 512), (1, 16392, 512), (1, 10000, 768), (1, 8200, 1024),
                                   (1, 16384, 1024), (1, 12296, 1536), (1, 14336, 1536), (1, 18432, 1536), (1, 16392, 2048),
                                   (1, 32768, 2048), (1, 32776, 2048), (1, 65536, 4080), (2, 8192, 512), (2, 8200, 512), (4, 4104, 1024)])
def test_quantize_gemm_is_the_two_calls(M, N, K):
    g = gen(N + K)
    x, B, SB = rows(g, M, K), codes(g, N, K), scales(g, R.blocks(N), R.blocks(K))
    bias = torch.randn(N, generator=g, device=DEV).to(torch.bfloat16)
    q, s = bs.fp8_quantize(x)
    assert torch.equal(bs.fp8_quantize_gemm(x, B, SB), bs.fp8_gemm(q, s, B, SB))
    assert torch.equal(bs.fp8_quantize_gemm(x, B, SB, bias=bias), bs.fp8_gemm(q, s, B, SB, bias=bias))
