"""64-bit references of the 8-bit products, the gated product and the block norms (test infrastructure),
and the error bounds their GPU results are held to.

Bounds count roundings: bf16 results are off by at most half a step (2^-8 of the value), binary32 operations by
2^-24 each.  A sum of K terms in binary32, in any order, is off by at most K 2^-24 sum|terms| when every addition
rounds to nearest; the matrix cores' additions may truncate, which doubles that.
"""
import math

import torch

BF = 2.0 ** -8
F32 = 2.0 ** -24


def act(name, g):
    """act(g) and act'(g), 64-bit."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(8 / math.pi)
    s = torch.sigmoid(k * (g + 0.044715 * g ** 3))
    return g * s, s + g * s * (1 - s) * k * (1 + 3 * 0.044715 * g ** 2)


#: 1 / (1 + 2^v) beyond the binary32 range (v > 126, where the sum or its reciprocal leaves the normal numbers) is 0
#: in the hardware's arithmetic and at most 2^-126 in truth: that much a sigmoid may be off in absolute terms, twice
#: that with the product around it.
UNDERFLOW = 2.0 ** -125


def act_slack(g):
    """Relative error of the binary32 activations in units of 2^-24: a few units of the hardware exp2 and
    reciprocal, and the rounding of their argument, which the exponential multiplies by the argument's size
    (2 g for the sigmoid, g^2 for erfc, g + g^3 with five roundings for the tanh form)."""
    return 32 + 8 * g.abs() + g * g + g.abs() ** 3


def int8_rows(x):
    """(codes, scales) of bf16 rows, by exact comparison of rationals: q is the even-rounded 127 x / amax."""
    xd = x.double()
    amax = xd.abs().amax(dim=1, keepdim=True) if x.shape[1] else xd.sum(1, keepdim=True)
    t = 127 * xd
    q = torch.where(amax > 0, torch.round(t / torch.where(amax > 0, amax, 1.0)), 0.0)
    # exact: |2 t - (2 q +- 1) amax| decides, all products exact in 53 bits
    assert bool(((2 * t - 2 * q * amax).abs() <= amax).all())
    tie = (2 * t - 2 * q * amax).abs() == amax
    assert bool((~tie | (amax == 0) | (q.remainder(2) == 0)).all())
    return q.to(torch.int8), (amax[:, 0].float() / torch.tensor(127.0, device=x.device))


def check(got, ref, slack, what):
    """|got - ref| <= 2^-8 |ref| + slack, elementwise, for a bf16 result."""
    bound = BF * ref.abs() + slack + 1e-40
    err = (got.double() - ref).abs()
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: error is {worst:.3f} of its bound"


def int8_product(A, SA, B, SB):
    return (A.double() @ B.double().t()) * SA.double()[:, None] * SB.double()[None, :]


def gated_check(h, G, U, eG, eU, name, what):
    """h against act(G) U, G and U known up to eG and eU."""
    a, da = act(name, G)
    # act' of any of the three is below 1.13 in magnitude
    slack = U.abs() * (1.13 * eG + act_slack(G) * F32 * a.abs() + G.abs() * UNDERFLOW) + a.abs() * eU + 1.13 * eG * eU + 4 * F32 * (a * U).abs()
    check(h, a * U, slack, what)


def rstd(v, eps):
    return 1.0 / torch.sqrt((v.double() ** 2).mean(dim=1, keepdim=True) + eps)


def norm_steps(x, residual, w_post, w_pre, gate, scale, eps):
    """The documented binary32 steps of block_norm (mean squares in 64 bits): (res, z) in bf16."""
    res = residual
    if x is not None:
        n = x.float() if w_post is None else x.float() * rstd(x, eps).float() * w_post.float()
        s32 = torch.tensor(scale, dtype=torch.float32, device=residual.device)
        g = s32
        if gate is not None:
            rows = gate.reshape(-1, residual.shape[1])
            g = rows.float().repeat_interleave(residual.shape[0] // rows.shape[0], dim=0) * s32
        res = (residual.float() + g * n).to(torch.bfloat16)
    if w_pre is None:
        return res, None
    return res, (res.float() * rstd(res, eps).float() * w_pre.float()).to(torch.bfloat16)


def norm64(x, residual, w_post, gate, scale, eps):
    """residual + gate scale n in 64 bits (inputs 64-bit)."""
    n = x if w_post is None else x / torch.sqrt((x * x).mean(dim=1, keepdim=True) + eps) * w_post
    g = scale
    if gate is not None:
        rows = gate.reshape(-1, residual.shape[1])
        g = rows.repeat_interleave(residual.shape[0] // rows.shape[0], dim=0) * scale
    return residual + g * n
