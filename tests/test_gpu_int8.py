"""GPU: the 8-bit quantiser and products against 64-bit references."""
import pytest
import torch

import block_scaled_fp4_e2m1_amd as bs
import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def rows(g, M, K, std=1.0):
    x = torch.randn((M, K), generator=g, device=DEV) * std
    x[:, :: max(1, K // 7)] *= 9
    return x.to(torch.bfloat16)


def codes(g, N, K):
    return torch.randint(-128, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)


@pytest.mark.parametrize("M,K", [(1, 8), (3, 64), (5, 2048), (2, 2056), (7, 8192), (1, 8200), (3, 32768), (2, 40008),
                                 (1, 131056), (1030, 520), (257, 7168)])
def test_quantise_exact(M, K):
    x = rows(gen(K + M), M, K)
    q, s = bs.int8_quantize(x)
    wq, ws = R.int8_rows(x)
    assert torch.equal(q, wq) and torch.equal(s, ws)


def test_quantise_every_tie():
    """Every bf16 value against every row maximum of one binade: all quotients that fall half-way between two
    integers are among them (the quotient depends on the significands and the exponents' difference only)."""
    amax = (0x3F80 + torch.arange(128, dtype=torch.int32)).to(torch.int16).view(torch.bfloat16)  # [1, 2)
    vals = (0x3B80 + torch.arange(0, 0x400, dtype=torch.int32)).to(torch.int16).view(torch.bfloat16)
    vals = vals[None, :].expand(128, -1).clone()
    vals[vals.float() > amax.float()[:, None]] = 0.0
    x = torch.cat([vals, -vals, amax[:, None], torch.zeros(128, 7, dtype=torch.bfloat16)], dim=1).to(DEV)
    q, s = bs.int8_quantize(x.contiguous())
    wq, ws = R.int8_rows(x)
    assert torch.equal(q, wq) and torch.equal(s, ws)


@pytest.mark.parametrize("power", [-132, -126, -100, -61, -60, -59, 59, 60, 61, 100, 126])
def test_quantise_extreme_scales(power):
    x = (torch.randn((4, 96), generator=gen(7), device=DEV, dtype=torch.float64) * 2.0 ** power).to(torch.bfloat16)
    q, s = bs.int8_quantize(x)
    wq, ws = R.int8_rows(x)
    assert torch.equal(q, wq) and torch.equal(s, ws)


def test_quantise_zero_and_nonfinite_rows():
    x = rows(gen(1), 6, 64)
    x[1] = 0.0
    x[2] = -0.0
    x[3, 5] = float("inf")
    x[4, 63] = float("nan")
    q, s = bs.int8_quantize(x)
    wq, ws = R.int8_rows(x[[0, 5]])
    assert torch.equal(q[[0, 5]], wq) and torch.equal(s[[0, 5]], ws)
    assert (q[1:5] == 0).all() and (s[1:3] == 0).all() and s[3:5].isnan().all()
    w, sw = codes(gen(2), 32, 64), torch.full((32,), 0.01, device=DEV)
    d = bs.int8_quantize_gemm(x, w, sw)
    assert (d[1:3] == 0).all() and d[3:5].isnan().all() and d[[0, 5]].isfinite().all()


SHAPES = [(1, 8, 16), (1, 4096, 7168), (2, 72, 48), (4, 256, 16384), (5, 520, 4096), (16, 1000, 2064), (17, 264, 512),
          (31, 128, 4112), (33, 8, 131056), (64, 512, 1040), (65, 648, 528), (130, 4096, 7168), (250, 1544, 4096),
          (300, 2048, 144), (513, 776, 2000), (1003, 512, 4096)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("with_bias", [False, True])
def test_gemm(M, N, K, with_bias):
    g = gen(M * 7 + N + K)
    A, B = codes(g, M, K), codes(g, N, K)
    SA = torch.rand(M, generator=g, device=DEV) + 0.01
    SB = (torch.rand(N, generator=g, device=DEV) + 0.01) * 1e-2
    bias = torch.randn(N, generator=g, device=DEV).to(torch.bfloat16) * 100 if with_bias else None
    guard = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
    out = bs.int8_gemm(A, SA, B, SB, bias=bias, out=guard[1:M + 1])
    ref = R.int8_product(A, SA, B, SB)
    # the integer sum is exact; its conversion, two products and the bias sum round once each
    slack = 3 * R.F32 * ref.abs()
    if bias is not None:
        slack = slack + R.F32 * (ref.abs() + bias.double().abs())
        ref = ref + bias.double()
    R.check(out, ref, 1.001 * slack, f"{M}x{N}x{K}")
    assert (guard[0] == 7).all() and (guard[M + 1] == 7).all()
    assert torch.equal(out, bs.int8_gemm(A, SA, B, SB, bias=bias))


def test_gemm_largest_sum():
    """All codes -128: the sum 2^14 K is the largest there is."""
    K = 131056
    A = torch.full((3, K), -128, dtype=torch.int8, device=DEV)
    B = torch.full((16, K), -128, dtype=torch.int8, device=DEV)
    B[1::2] = 127
    one = lambda n: torch.ones(n, device=DEV)  # noqa: E731
    d = bs.int8_gemm(A, one(3), B, one(16)).double()
    for c, v in ((0, 128 * 128 * K), (1, -128 * 127 * K)):
        assert ((d[:, c::2] - v).abs() <= (R.BF + R.F32) * abs(v)).all()


@pytest.mark.parametrize("M,N,K", [(1, 4096, 7168), (1, 136, 16), (2, 520, 1040), (3, 512, 8192), (4, 96, 16384),
                                   (4, 64, 16400), (5, 256, 512), (16, 512, 2048), (40, 264, 7168), (200, 512, 4096),
                                   (1, 264, 9472), (1, 520, 9344), (2, 72, 4720), (4, 136, 2320), (4, 40, 2384),
                                   (3, 8, 48), (4, 7168, 4096)])
def test_quantize_gemm_is_the_two_calls(M, N, K):
    g = gen(N + K)
    x = rows(g, M, K)
    if M > 1:
        x[M - 1] = 0.0
    B, SB = codes(g, N, K), torch.rand(N, generator=g, device=DEV)
    bias = torch.randn(N, generator=g, device=DEV).to(torch.bfloat16)
    want = bs.int8_gemm(*bs.int8_quantize(x), B, SB, bias=bias)
    assert torch.equal(bs.int8_quantize_gemm(x, B, SB, bias=bias), want)
    assert torch.equal(bs.int8_quantize_gemm(x, B, SB), bs.int8_gemm(*bs.int8_quantize(x), B, SB))


@pytest.mark.parametrize("M,I,K", [(1, 8, 16), (1, 768, 2048), (5, 7168, 4096), (16, 264, 1040), (19, 72, 512),
                                   (64, 520, 2064), (70, 1544, 528), (333, 776, 2048), (600, 2048, 256)])
@pytest.mark.parametrize("act", sorted(bs.ACTIVATIONS))
def test_gated(M, I, K, act):
    g = gen(M + I + K)
    A, W = codes(g, M, K), codes(g, 2 * I, K)
    SA = (torch.rand(M, generator=g, device=DEV) + 0.5) * 0.02
    SW = (torch.rand(2 * I, generator=g, device=DEV) + 0.5) * 0.02 / K ** 0.5
    h = bs.int8_gated_ffn(A, SA, W, SW, act=act)
    y = R.int8_product(A, SA, W, SW)
    G, U = y[:, :I], y[:, I:]
    R.gated_check(h, G, U, 3.1 * R.F32 * G.abs(), 3.1 * R.F32 * U.abs(), act, f"{M}x{I}x{K} {act}")
    assert torch.equal(h, bs.int8_gated_ffn(A, SA, W, SW, act=act))


def test_gated_wide_range():
    """Gates from deep in the negative tail to large values."""
    M, I, K = 40, 256, 64
    A = torch.zeros((M, K), dtype=torch.int8, device=DEV)
    A[:, 0] = torch.arange(M, device=DEV).to(torch.int8) - 20
    A[:, 1] = 64
    W = torch.zeros((2 * I, K), dtype=torch.int8, device=DEV)
    W[:I, 0] = torch.arange(I, device=DEV).sub(128).to(torch.int8)
    W[I:, 1] = 100
    SA = torch.full((M,), 0.1, device=DEV)
    SW = torch.full((2 * I,), 0.1, device=DEV)
    y = R.int8_product(A, SA, W, SW)
    for act in bs.ACTIVATIONS:
        h = bs.int8_gated_ffn(A, SA, W, SW, act=act)
        R.gated_check(h, y[:, :I], y[:, I:], 3.1 * R.F32 * y[:, :I].abs(), 3.1 * R.F32 * y[:, I:].abs(), act, act)


def test_empty():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    W, SW = codes(gen(0), 32, 64), torch.ones(32, device=DEV)
    q, s = bs.int8_quantize(x)
    assert q.shape == (0, 64) and s.shape == (0,)
    assert bs.int8_gemm(q, s, W, SW).shape == (0, 32)
    assert bs.int8_quantize_gemm(x, W, SW).shape == (0, 32)
    assert bs.int8_gated_ffn(q, s, W, SW).shape == (0, 16)


@pytest.mark.parametrize("M,N,K", [(1, 16384, 512), (1, 16392, 512), (4, 4096, 1024), (4, 4104, 1024), (2, 16384, 4096),
                                   (2, 16392, 4096), (1, 40968, 2048)])
def test_quantize_gemm_at_the_width_limits(M, N, K):
    """Both sides of the widths up to which the rows are quantised in the product's workgroups."""
    g = gen(N + K)
    x, B, SB = rows(g, M, K), codes(g, N, K), torch.rand(N, generator=g, device=DEV)
    d = bs.int8_quantize_gemm(x, B, SB)
    q, s = R.int8_rows(x)
    ref = R.int8_product(q, s, B, SB)
    R.check(d, ref, 3.1 * R.F32 * ref.abs(), f"{M}x{N}x{K}")
    assert torch.equal(d, bs.int8_gemm(*bs.int8_quantize(x), B, SB))


def test_quantize_gemm_very_wide():
    """2^27 columns: 32 threads for each would be more than a launch can hold."""
    N, K = (1 << 27) + 8, 16
    g = gen(3)
    x, B, SB = rows(g, 1, K), codes(g, N, K), torch.rand(N, generator=g, device=DEV)
    d = bs.int8_quantize_gemm(x, B, SB)
    c = torch.cat([torch.arange(512, device=DEV), torch.arange(N - 512, N, device=DEV)])
    q, s = R.int8_rows(x)
    ref = R.int8_product(q, s, B[c], SB[c])
    R.check(d[:, c], ref, 3.1 * R.F32 * ref.abs(), "d")
    assert torch.equal(d, bs.int8_gemm(q, s, B, SB))


def one_call(M, N, K):
    """Whether int8_quantize_gemm is one launch (no workspace), so that a changed rule cannot empty the tests below."""
    from block_scaled_fp4_e2m1_amd import binding
    return binding.load().bsfp4_int8_quantize_gemm_workspace_size(M, N, K) == 0


@pytest.mark.parametrize("M,K,one", [(1, 9216, True), (1, 9232, False), (2, 4608, True), (2, 4624, False),
                                     (3, 3056, True), (3, 3088, False), (4, 2304, True), (4, 2320, False),
                                     (4, 2032, True), (3, 1008, True), (2, 2320, True), (1, 8208, True), (4, 16, True)])
@pytest.mark.parametrize("N", [8, 520, 1000])
def test_quantise_in_the_product(M, K, one, N):
    """Rows quantised inside the product's workgroups, up to a full LDS area, against 64 bits and the two calls."""
    assert one_call(M, N, K) == one
    g = gen(M + N + K)
    x = rows(g, M, K)
    B, SB = codes(g, N, K), torch.rand(N, generator=g, device=DEV) + 0.01
    bias = torch.randn(N, generator=g, device=DEV).to(torch.bfloat16) * 100
    guard = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
    d = bs.int8_quantize_gemm(x, B, SB, bias=bias, out=guard[1:M + 1])
    q, s = R.int8_rows(x)
    ref = R.int8_product(q, s, B, SB)
    slack = 3 * R.F32 * ref.abs() + R.F32 * (ref.abs() + bias.double().abs())
    R.check(d, ref + bias.double(), 1.001 * slack, f"{M}x{N}x{K}")
    assert (guard[0] == 7).all() and (guard[M + 1] == 7).all()
    assert torch.equal(d, bs.int8_gemm(*bs.int8_quantize(x), B, SB, bias=bias))


@pytest.mark.parametrize("M,K", [(1, 9216), (2, 4608), (3, 3056), (4, 2304), (4, 112)])
@pytest.mark.parametrize("row", [0, -1])
@pytest.mark.parametrize("value", [0.0, float("inf"), float("-inf"), float("nan")])
def test_quantise_in_the_product_degenerate_rows(M, K, row, value):
    """A row of zeros gives zeros (the bias), one infinity or NaN, wherever in the row, a row of NaN; the rows beside
    it are what they are without it."""
    N = 136
    assert one_call(M, N, K)
    g = gen(M + K)
    x, B, SB = rows(g, M, K), codes(g, N, K), torch.rand(N, generator=g, device=DEV) + 0.01
    bias = torch.randn(N, generator=g, device=DEV).to(torch.bfloat16)
    want = bs.int8_quantize_gemm(x, B, SB, bias=bias)
    for at in (0, K // 2 + 3, K - 1):
        y = x.clone()
        if value == 0.0:
            y[row] = 0.0
        else:
            y[row, at] = value
        d = bs.int8_quantize_gemm(y, B, SB, bias=bias)
        others = [m for m in range(M) if m != row % M]
        assert torch.equal(d[others], want[others])
        assert torch.equal(d[row], bias) if value == 0.0 else d[row].isnan().all()
