"""GPU: the matrix products of the block operators through every tile kernel, K split and part launch that the plan
takes on 256 compute units, and over operands whose bytes pass 32 bits, against 64-bit references."""
import pytest
import torch

import block_scaled_fp4_e2m1_amd as bs
import block_ref as R
from test_gpu_gated_ffn import backward_reference, problem, sum_error

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

#: rows, weight rows (gated: both halves), bytes of a row
SHAPES = {
    "128": (336, 6160, 288), "128 cols+64": (80, 68768, 1472), "128 cols+64x128": (80, 79056, 1216),
    "128 rows+64": (2064, 4336, 1024), "128 split": (80, 11024, 11040), "deep": (336, 6160, 2080),
    "deep split": (80, 6160, 8224), "256": (5008, 6160, 288), "256 cols+deep": (2512, 14352, 2080),
    "256 cols+256x128": (5008, 14352, 2080), "256 cols+128": (640, 34320, 1280), "256 cols+64": (4096, 4112, 2080),
    "256 rows+256x128": (5008, 4112, 8224), "256 rows+128": (640, 95120, 320), "256 rows+64": (2064, 14352, 2080),
    "256 split": (144, 12000, 12704), "256x128": (2064, 14352, 288), "256x128 cols+64": (208, 33744, 928),
    "256x128 rows+64": (5008, 1552, 2080), "256x128 rows+64x128": (2064, 4112, 8224),
    "256x128 split": (144, 5568, 9216), "64": (80, 272, 288), "64 split": (80, 272, 8224), "64x128": (80, 10256, 2080),
    "64x128 split": (80, 2064, 8224),
}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def int8_problem(M, N, K):
    g = gen(M + N + K)
    code = lambda *s: torch.randint(-128, 128, s, generator=g, device=DEV, dtype=torch.int8)  # noqa: E731
    return (code(M, K), (torch.rand(M, generator=g, device=DEV) + 0.5) * 0.02, code(N, K),
            (torch.rand(N, generator=g, device=DEV) + 0.5) * 0.02 / K ** 0.5)


@pytest.mark.parametrize("kind", SHAPES)
def test_int8_gemm(kind):
    M, N, K = SHAPES[kind]
    M -= 3
    A, SA, B, SB = int8_problem(M, N, K)
    guard = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
    out = bs.int8_gemm(A, SA, B, SB, out=guard[1:M + 1])
    ref = R.int8_product(A, SA, B, SB)
    R.check(out, ref, 3.1 * R.F32 * ref.abs(), kind)
    assert (guard[0] == 7).all() and (guard[M + 1] == 7).all()


@pytest.mark.parametrize("kind", SHAPES)
def test_int8_gated(kind):
    M, N, K = SHAPES[kind]
    M, I = M - 1, N // 2
    A, SA, W, SW = int8_problem(M, N, K)
    guard = torch.full((M + 2, I), 7.0, dtype=torch.bfloat16, device=DEV)
    h = bs.int8_gated_ffn(A, SA, W, SW, out=guard[1:M + 1])
    y = R.int8_product(A, SA, W, SW)
    R.gated_check(h, y[:, :I], y[:, I:], 3.1 * R.F32 * y[:, :I].abs(), 3.1 * R.F32 * y[:, I:].abs(), "silu", kind)
    assert (guard[0] == 7).all() and (guard[M + 1] == 7).all()


@pytest.mark.parametrize("kind", SHAPES)
def test_gated(kind):
    M, N, kbytes = SHAPES[kind]
    M, I, H = M - 2, N // 2, kbytes // 2
    x, W, _ = problem(M, H, I)
    y, e = x.double() @ W.double().t(), sum_error(x, W)
    guard = torch.full((M + 2, I), 7.0, dtype=torch.bfloat16, device=DEV)
    h = bs.gated_ffn(x, W, out=guard[1:M + 1])
    R.gated_check(h, y[:, :I], y[:, I:], e[:, :I], e[:, I:], "silu", kind)
    assert (guard[0] == 7).all() and (guard[M + 1] == 7).all()
    h2, gu = bs.gated_ffn(x, W, save_gate_up=True)
    assert torch.equal(h2, h) and ((gu.double() - y).abs() <= e).all()


@pytest.mark.parametrize("kind", SHAPES)
@pytest.mark.parametrize("which", ["dx", "dW"])
def test_gradients(kind, which):
    """dx = [dG | dU] @ W13 sums over the weight's rows, dW13 = [dG | dU]^T @ x over the tokens."""
    rows, H, kbytes = SHAPES[kind]
    M, I = (rows - 3, kbytes // 4) if which == "dx" else (kbytes // 2, rows // 2)
    x, W, dh = problem(M, H, I)
    gu = torch.randn((M, 2 * I), generator=gen(M), device=DEV) * 2
    dx, dW = bs.gated_ffn_backward(dh, x, W, gu, need_dx=which == "dx", need_dW13=which == "dW")
    rx, rw, sx, sw = backward_reference(dh, x, W, gu, "silu")
    R.check(dx if which == "dx" else dW, *((rx, sx) if which == "dx" else (rw, sw)), f"{which} {kind}")


# ---- operands of more than 2^32 bytes: the first, the last and the rows around the passes are checked

def spots(n, row_bytes):
    """Rows at both ends and around every 2^31st byte."""
    s = set(range(3)) | set(range(n - 3, n))
    for k in range(1, n * row_bytes // 2 ** 31 + 1):
        at = k * 2 ** 31 // row_bytes
        s |= {r for r in range(at - 2, at + 3) if 0 <= r < n}
    return torch.tensor(sorted(s), device=DEV)


def big_bf16(rows, cols, std, seed):
    t = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    g = gen(seed)
    for a in range(0, rows, 1 << 15):
        b = t[a:a + (1 << 15)]
        b.copy_(torch.randn(b.shape, generator=g, device=DEV) * std)
    return t


@pytest.mark.parametrize("M", [1, 11, 140])
def test_large_gated_weight(M):
    """A weight of 5.4 GB (its up half begins past 2^31 bytes): forward, and both gradients."""
    H, I = 8192, 163848
    W = big_bf16(2 * I, H, H ** -0.5, 1)
    x, dh = big_bf16(M, H, 1.0, 2), big_bf16(M, I, 1.0, 3)
    h, gu = bs.gated_ffn(x, W, save_gate_up=True)
    c = spots(I, 2 * H)
    Wc = torch.cat([W[c], W[I + c]])
    y, e, n = x.double() @ Wc.double().t(), sum_error(x, Wc), c.numel()
    R.gated_check(h[:, c], y[:, :n], y[:, n:], e[:, :n], e[:, n:], "silu", "h")
    assert torch.equal(bs.gated_ffn(x, W), h)
    assert ((gu[:, torch.cat([c, I + c])].double() - y).abs() <= e).all()
    dx, dW = bs.gated_ffn_backward(dh, x, W, gu)
    _, rw, _, sw = backward_reference(dh[:, c].contiguous(), x, Wc, torch.cat([gu[:, c], gu[:, I + c]], 1), "silu")
    R.check(dW[torch.cat([c, I + c])], rw, sw, "dW")
    k = spots(H, 1)
    rx, _, sx, _ = backward_reference(dh, x[:, k].contiguous(), W[:, k].contiguous(), gu, "silu")
    R.check(dx[:, k], rx, sx, "dx")


@pytest.mark.parametrize("N", [72, 1040])
def test_large_int8_batch(N):
    """600000 tokens: 4.9 GB of codes, 9.8 GB of bf16 rows, and the same through the fused call."""
    M, K = 600011, 8192
    x = big_bf16(M, K, 1.0, 4)
    q, s = bs.int8_quantize(x)
    r = spots(M, K)
    wq, ws = R.int8_rows(x[r])
    assert torch.equal(q[r], wq) and torch.equal(s[r], ws)
    _, _, B, SB = int8_problem(1, N, K)
    d = bs.int8_gemm(q, s, B, SB)
    ref = R.int8_product(q[r], s[r], B, SB)
    R.check(d[r], ref, 3.1 * R.F32 * ref.abs(), "d")
    I = N // 2 // 8 * 8
    h = bs.int8_gated_ffn(q, s, B[:2 * I], SB[:2 * I])
    R.gated_check(h[r], ref[:, :I], ref[:, I:2 * I], 3.1 * R.F32 * ref[:, :I].abs(), 3.1 * R.F32 * ref[:, I:2 * I].abs(),
                  "silu", "h")
    del q
    assert torch.equal(bs.int8_quantize_gemm(x, B, SB), d)


def test_large_training_batch():
    """400000 tokens of 6400: 5.1 GB of rows, and gate_up of 2.5 GB."""
    M, H, I = 400009, 6400, 776
    W, x, dh = big_bf16(2 * I, H, H ** -0.5, 5), big_bf16(M, H, 1.0, 6), big_bf16(M, I, 1.0, 7)
    h, gu = bs.gated_ffn(x, W, save_gate_up=True)
    r = spots(M, 2 * H)
    y, e = x[r].double() @ W.double().t(), sum_error(x[r], W)
    R.gated_check(h[r], y[:, :I], y[:, I:], e[:, :I], e[:, I:], "silu", "h")
    dx, dW = bs.gated_ffn_backward(dh, x, W, gu)
    rx, _, sx, _ = backward_reference(dh[r], x[r], W, gu[r], "silu")
    R.check(dx[r], rx, sx, "dx")
    k = spots(H, 1)
    _, rw, _, sw = backward_reference(dh, x[:, k].contiguous(), W[:, k].contiguous(), gu, "silu")
    R.check(dW[:, k], rw, sw, "dW")


def test_large_norm_batch():
    """300000 rows of 8192: 4.9 GB each; a gate for every 3 rows."""
    T, H, groups = 300000, 8192, 100000
    x, residual, gate = big_bf16(T, H, 1.0, 8), big_bf16(T, H, 3.0, 9), big_bf16(groups, H, 1.0, 10)
    w = big_bf16(2, H, 1.0, 11)
    kw = dict(w_post=w[0], w_pre=w[1], scale=0.4)
    res, z = bs.block_norm(x, residual, gate=gate, **kw)
    r = spots(T, 2 * H)
    # the checked rows with a gate each
    wres, wz = R.norm_steps(x[r], residual[r], w[0], w[1], gate[r // 3], 0.4, 1e-6)
    assert torch.equal(res[r], wres) and torch.equal(z[r], wz)
    _, q, s = bs.block_norm(x, residual, gate=gate, fmt="int8", **kw)
    wq, ws = R.int8_rows(wz)
    assert torch.equal(q[r], wq) and torch.equal(s[r], ws)
    del q, s, z
    dx, dr, _, _, dg = bs.block_norm_backward(residual, x, x, res, gate=gate, **kw)
    # rows and their gate's group do not depend on the others: the same groups alone give the same bits
    g = torch.unique(r // 3)
    rows = (g[:, None] * 3 + torch.arange(3, device=DEV)).flatten()
    dx2, dr2, _, _, dg2 = bs.block_norm_backward(residual[rows], x[rows], x[rows], res[rows], gate=gate[g], **kw)
    assert torch.equal(dx[rows], dx2) and torch.equal(dr[rows], dr2)
    assert ((dg[g] - dg2).abs() <= 8 * R.F32 * 3 * dg2.abs().max()).all()


def test_most_rows():
    """As many rows as a launch of the row kernels holds (2^26 - 4), of eight values each."""
    T, H = (1 << 26) - 4, 8
    x = big_bf16(T, H, 1.0, 12)
    w = big_bf16(1, H, 1.0, 13)[0]
    r = torch.cat([torch.arange(9, device=DEV), torch.arange(T - 9, T, device=DEV)])
    q, s = bs.int8_quantize(x)
    wq, ws = R.int8_rows(x[r])
    assert torch.equal(q[r], wq) and torch.equal(s[r], ws)
    _, z = bs.block_norm(None, x, w_pre=w)
    assert torch.equal(z[r], R.norm_steps(None, x[r], None, w, None, 1.0, 1e-6)[1])
    _, dr, _, dw, _ = bs.block_norm_backward(None, z, None, x, w_pre=w)
    _, dr2, _, _, _ = bs.block_norm_backward(None, z[r], None, x[r], w_pre=w)
    assert torch.equal(dr[r], dr2)
