"""CPU: which kernels the block operators' calls take, where tests or a launch's limits hang on it."""
import pytest

from block_scaled_fp4_e2m1_amd import binding


def fused(M, N, K):
    """Whether int8_quantize_gemm quantises inside the product's workgroups: it needs no workspace then."""
    return binding.load().bsfp4_int8_quantize_gemm_workspace_size(M, N, K) == 0


@pytest.mark.parametrize("M", [1, 2, 3, 4])
def test_fused_quantiser_by_rows(M):
    """Up to where the rows and their codes fit in LDS."""
    K = 9216 // M
    assert fused(M, 512, K) and not fused(M, 512, K + 16) and not fused(M + 1, 512, K)


@pytest.mark.parametrize("M,K,last", [(1, 512, 16384), (1, 1024, 16384), (1, 2048, 32768), (1, 4096, 131072),
                                      (2, 1024, 8192), (2, 4096, 16384), (3, 1024, 5456), (4, 2304, 4096)])
def test_fused_quantiser_by_columns(M, K, last):
    """Every workgroup quantises the rows again: past some width two launches take over."""
    assert fused(M, last, K) and not fused(M, last + 8, K)


def test_fused_quantiser_within_a_launch():
    """32 threads per column, fewer than 2^32 in a launch, for every width that is admitted."""
    assert not any(fused(M, 1 << p, K) for M in (1, 2, 3, 4) for p in range(27, 30) for K in range(16, 9217, 16))
