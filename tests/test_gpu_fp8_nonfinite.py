"""GPU: an E4M3 NaN code or a scale that is not finite spoils the results that are computed from it and no other, in every
kernel that a product or an expert layer takes."""
import pytest
import torch

import block_scaled_fp4_e2m1_amd as bs
import fp8_ref as R
from test_gpu_fp8_moe import DEV, F8, codes, gen, scales

pytestmark = pytest.mark.gpu
NAN = 0x7F  # an E4M3 NaN; 0xFF is the other


def put(t, at, code):
    t.view(torch.uint8)[at] = code


# tokens, hidden size, intermediate size, experts: quantised in the workgroups and apart, and past a handful
LAYERS = [(2, 256, 128, 6), (4, 272, 256, 6), (5, 1040, 128, 6), (8, 512, 384, 6), (64, 512, 384, 6), (600, 256, 128, 6)]


@pytest.mark.parametrize("T,H,I,E", LAYERS)
@pytest.mark.parametrize("what", ["W2", "W2s", "W13", "W13s"])
def test_layer_keeps_an_experts_nan_to_its_tokens(T, H, I, E, what):
    """Expert 1 is spoiled.  Tokens that do not meet it are bit for bit what they were; of those that do, only what a W2 code
    reaches is NaN."""
    g = gen(T + H + I)
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    ids = torch.randint(2, E, (T, 2), generator=g, device=DEV, dtype=torch.int32)
    ids[:, 1] = torch.where(ids[:, 1] == ids[:, 0], 0, ids[:, 1])
    ids[0, 0] = -1  # the first pair's row is never written
    ids[T - 1, 1] = 1
    if T > 4:
        ids[3] = torch.tensor([1, 1], dtype=torch.int32)  # twice
        ids[2] = -1  # a token of no expert
    meets = (ids == 1).any(1)
    w = torch.rand((T, 2), generator=g, device=DEV) + 0.1
    W13, W13s = codes(g, E, 2 * I, H), scales(g, E, R.blocks(2 * I), R.blocks(H)) * 0.02
    W2, W2s = codes(g, E, H, I), scales(g, E, R.blocks(H), R.blocks(I)) * 0.02
    good = bs.fp8_moe_layer(x, ids, w, W13, W13s, W2, W2s)
    assert good.isfinite().all()
    nan = torch.zeros(H, dtype=torch.bool, device=DEV)
    if what == "W2":
        for n, k, code in ((0, 0, NAN), (H - 1, I - 1, 0xFF), (H // 2 + 3, I // 2, NAN)):
            put(W2, (1, n, k), code)
            nan[n] = True
    elif what == "W2s":
        W2s[1, 0, 0], nan[:R.BLOCK] = float("nan"), True
        W2s[1, R.blocks(H) - 1, R.blocks(I) - 1] = float("inf")
        nan[(R.blocks(H) - 1) * R.BLOCK:] = True  # an infinity or, where the code is zero, a NaN
    elif what == "W13":
        put(W13, (1, I + 5, H - 1), NAN)
        nan[:] = True  # the block's scale is NaN
    else:
        W13s[1, 0, 0], nan[:] = float("nan"), True
    out = bs.fp8_moe_layer(x, ids, w, W13, W13s, W2, W2s)
    assert torch.equal(out[~meets], good[~meets])
    assert not out[meets][:, nan].isfinite().any()
    assert torch.equal(out[meets][:, ~nan], good[meets][:, ~nan])


@pytest.mark.parametrize("M,N,K", [(1, 264, 272), (4, 136, 2064), (12, 264, 528), (30, 136, 528), (100, 264, 272), (300, 1040, 2064)])
@pytest.mark.parametrize("by_row", [False, True])
def test_product_keeps_a_nan_to_its_row_and_column(M, N, K, by_row):
    g = gen(M + N + K)
    A, B = codes(g, M, K), codes(g, N, K)
    SA, SB = scales(g, R.blocks(K), M), scales(g, *((R.blocks(K), N) if by_row else (R.blocks(N), R.blocks(K))))
    good = bs.fp8_gemm(A, SA, B, SB)
    m, n = M // 2, N - 3
    put(A, (m, K - 1), NAN)
    put(B, (n, 0), 0xFF)
    out = bs.fp8_gemm(A, SA, B, SB)
    want = good.clone()
    want[m], want[:, n] = float("nan"), float("nan")
    assert torch.equal(out.isnan(), want.isnan()) and torch.equal(out.nan_to_num(), want.nan_to_num())
