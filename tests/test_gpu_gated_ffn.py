"""GPU: the gated feed-forward product in bf16, forward and backward, against 64-bit references."""
import pytest
import torch

import block_scaled_fp4_e2m1_amd as bs
import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ACTS = sorted(bs.ACTIVATIONS)


def problem(M, H, I, seed=0, wstd=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + M + 3 * H + 5 * I)
    bf = lambda *s, std=1.0: (torch.randn(s, generator=g, device=DEV) * std).to(torch.bfloat16)  # noqa: E731
    return bf(M, H), bf(2 * I, H, std=wstd or 1.5 / H ** 0.5), bf(M, I)


def sum_error(a, b):
    """Bound of a binary32 sum of products a @ b^T (exact products, 2 K 2^-24 of the absolute sum)."""
    return 2 * (a.shape[1] + 8) * R.F32 * (a.double().abs() @ b.double().abs().t())


SHAPES = [(1, 8, 8), (1, 4096, 7168), (2, 264, 72), (9, 2048, 768), (16, 520, 1544), (17, 128, 256), (40, 1000, 264),
          (64, 2048, 512), (100, 72, 776), (257, 512, 1032), (333, 2048, 1544), (777, 1032, 520)]


@pytest.mark.parametrize("M,H,I", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_forward(M, H, I, act):
    x, W, _ = problem(M, H, I)
    y = x.double() @ W.double().t()
    e = sum_error(x, W)
    G, U = y[:, :I], y[:, I:]
    guard = torch.full((M + 2, I), 7.0, dtype=torch.bfloat16, device=DEV)
    h = bs.gated_ffn(x, W, act=act, out=guard[1:M + 1])
    R.gated_check(h, G, U, e[:, :I], e[:, I:], act, f"h {M}x{H}x{I}")
    assert (guard[0] == 7).all() and (guard[M + 1] == 7).all()
    h2, gu = bs.gated_ffn(x, W, act=act, save_gate_up=True)
    assert torch.equal(h2, h)
    assert gu.dtype == torch.float32 and ((gu.double() - y).abs() <= e).all()


def backward_reference(dh, x, W, gate_up, act):
    """(dx, dW) in 64 bits from the saved gate_up, and bounds beyond their own rounding: [dG | dU] is rounded to
    bf16 (2^-8 of each) after a handful of binary32 steps."""
    I = dh.shape[1]
    G, U, d = gate_up[:, :I].double(), gate_up[:, I:].double(), dh.double()
    a, da = R.act(act, G)
    dgu = torch.cat([d * U * da, d * a], dim=1)
    # act' has the activations' relative error on each of its two terms, both at most 1.13 + |G|
    e = torch.cat([(d * U).abs() * (1.13 + G.abs()) * R.act_slack(G) * R.F32,
                   d.abs() * a.abs() * R.act_slack(G) * R.F32], dim=1) + R.BF * 1.01 * dgu.abs()
    # a sigmoid below the normal binary32 numbers is 0: act' = s (1 + G (1 - s)) and act = G s lose that much
    e = e + R.UNDERFLOW * torch.cat([(d * U).abs() * (1 + G.abs()), d.abs() * G.abs()], dim=1)
    Wd, xd = W.double(), x.double()
    big = dgu.abs() + e
    dx, dW = dgu @ Wd, dgu.t() @ xd
    sx = e @ Wd.abs() + 2 * (2 * I + 8) * R.F32 * (big @ Wd.abs())
    sw = e.t() @ xd.abs() + 2 * (dh.shape[0] + 8) * R.F32 * (big.t() @ xd.abs())
    return dx, dW, sx, sw


@pytest.mark.parametrize("M,H,I", [(1, 8, 8), (3, 72, 40), (15, 256, 128), (63, 264, 72), (64, 512, 256),
                                   (65, 1032, 264), (200, 2048, 776), (513, 520, 1544), (777, 2048, 768),
                                   (1024, 1024, 1024), (256, 4096, 1024), (4096, 512, 1024), (1500, 2056, 1000)])
@pytest.mark.parametrize("act", ACTS)
def test_backward(M, H, I, act):
    x, W, dh = problem(M, H, I, seed=1)
    _, gu = bs.gated_ffn(x, W, act=act, save_gate_up=True)
    dx, dW = bs.gated_ffn_backward(dh, x, W, gu, act=act)
    rx, rw, sx, sw = backward_reference(dh, x, W, gu, act)
    R.check(dx, rx, sx, f"dx {M}x{H}x{I}")
    R.check(dW, rw, sw, f"dW {M}x{H}x{I}")
    dx2, none = bs.gated_ffn_backward(dh, x, W, gu, act=act, need_dW13=False)
    assert none is None and torch.equal(dx, dx2)
    none, dW2 = bs.gated_ffn_backward(dh, x, W, gu, act=act, need_dx=False)
    assert none is None and torch.equal(dW, dW2)


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """Directional derivatives of L = sum(h dh) by central differences of the 64-bit function.  The difference has
    error O(t^2); the gradients' is that of bf16 operands, averaged over the sum: 1 % of the gradient's norm along
    a random direction of unit elements is far above both (2^-8 per term, random signs)."""
    M, H, I = 48, 128, 96
    x, W, dh = problem(M, H, I, seed=2)
    _, gu = bs.gated_ffn(x, W, act=act, save_gate_up=True)
    dx, dW = bs.gated_ffn_backward(dh, x, W, gu, act=act)

    def loss(xx, ww):
        y = xx @ ww.t()
        return (R.act(act, y[:, :I])[0] * y[:, I:] * dh.double()).sum()

    t = 1e-4
    for grad, (ex, ew) in ((dx, (1.0, 0.0)), (dW, (0.0, 1.0))):
        base = x if ex else W
        E = torch.randn(base.shape, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV, dtype=torch.float64)
        xp, wp = x.double(), W.double()
        diff = (loss(xp + t * ex * E if ex else xp, wp + t * ew * E if ew else wp) -
                loss(xp - t * ex * E if ex else xp, wp - t * ew * E if ew else wp)) / (2 * t)
        got = (grad.double() * E).sum()
        assert (got - diff).abs() <= 1e-2 * grad.double().norm(), (act, got.item(), diff.item())


def test_extreme_gates():
    """Gates far out in both tails, infinite products included, give no NaN in h where the 64-bit form has none."""
    M, H, I = 8, 16, 64
    x = torch.zeros((M, H), dtype=torch.bfloat16, device=DEV)
    x[:, 0] = torch.tensor([-1e4, -100.0, -12.0, -1.0, 0.0, 1.0, 100.0, 1e4], device=DEV).to(torch.bfloat16)
    x[:, 1] = 1.0
    W = torch.zeros((2 * I, H), dtype=torch.bfloat16, device=DEV)
    W[:I, 0] = 1.0
    W[I:, 1] = 2.0
    dh = torch.ones((M, I), dtype=torch.bfloat16, device=DEV)
    for act in ACTS:
        h, gu = bs.gated_ffn(x, W, act=act, save_gate_up=True)
        G, U = gu[:, :I].double(), gu[:, I:].double()
        R.gated_check(h, G, U, 0.0 * G, 0.0 * U, act, act)
        dx, dW = bs.gated_ffn_backward(dh, x, W, gu, act=act)
        rx, rw, sx, sw = backward_reference(dh, x, W, gu, act)
        R.check(dx, rx, sx, act)
        R.check(dW, rw, sw, act)


def test_empty_batch():
    x, W, dh = problem(4, 64, 32)
    h, gu = bs.gated_ffn(x[:0], W, save_gate_up=True)
    assert h.shape == (0, 32) and gu.shape == (0, 64)
    dx, dW = bs.gated_ffn_backward(dh[:0], x[:0], W, gu)
    assert dx.shape == (0, 64) and dW.shape == W.shape and (dW == 0).all()
