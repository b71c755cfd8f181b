"""GPU: the norms around a block, forward and backward."""
import pytest
import torch

import block_scaled_fp4_e2m1_amd as bs
import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6


def problem(T, H, groups, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + T + H)
    bf = lambda *s, std=1.0, mean=0.0: (torch.randn(s, generator=g, device=DEV) * std + mean).to(torch.bfloat16)  # noqa: E731
    p = dict(x=bf(T, H), residual=bf(T, H, std=3.0), w_post=bf(H, std=0.2, mean=1.0), w_pre=bf(H, std=0.2, mean=1.0),
             gate=None if groups == 0 else bf(H) if groups == -1 else bf(groups, H))
    return p, bf(T, H), bf(T, H)


SHAPES = [(1, 8, 0), (1, 4096, 1), (3, 16, 3), (5, 504, 1), (4, 512, -1), (7, 520, 7), (6, 1032, 2), (9, 2048, 3),
          (33, 2056, 0), (12, 4096, 4), (5, 4104, -1), (3, 7168, 1), (4, 8192, 2), (3, 8200, 1), (2, 16384, 2),
          (700, 264, 7), (1024, 1024, -1), (2000, 136, 2000)]


@pytest.mark.parametrize("T,H,groups", SHAPES)
@pytest.mark.parametrize("parts", ["all", "no_post", "no_pre", "pre_only"])
def test_forward_bytes(T, H, groups, parts):
    """The documented steps, bit for bit, and each within its roundings of the 64-bit value."""
    p, _, _ = problem(T, H, groups)
    if parts == "no_post":
        p["w_post"] = None
    if parts == "no_pre":
        p["w_pre"] = None
    if parts == "pre_only":
        p["x"] = p["w_post"] = p["gate"] = None
    kw = dict(w_post=p["w_post"], w_pre=p["w_pre"], gate=p["gate"], scale=0.3, eps=EPS)
    got = bs.block_norm(p["x"], p["residual"], **kw)
    res, z = got if p["w_pre"] is not None else (got, None)
    wres, wz = R.norm_steps(p["x"], p["residual"], p["w_post"], p["w_pre"], p["gate"], 0.3, EPS)
    assert torch.equal(res, wres)
    if p["x"] is not None:
        d = lambda t: None if t is None else t.double()  # noqa: E731
        ref = R.norm64(d(p["x"]), d(p["residual"]), d(p["w_post"]), d(p["gate"]), 0.3, EPS)
        # rstd, two products, gate * scale, its product, the sum: 6 roundings of the two terms
        R.check(res, ref, 8 * R.F32 * (p["residual"].double().abs() + (ref - p["residual"].double()).abs()), "res")
    if z is None:
        return
    assert torch.equal(z, wz)
    ref = res.double() * R.rstd(res, EPS) * p["w_pre"].double()
    R.check(z, ref, 4 * R.F32 * ref.abs(), "z")
    res8, q, s = bs.block_norm(p["x"], p["residual"], fmt="int8", **kw)
    wq, ws = bs.int8_quantize(z)
    assert torch.equal(res8, res) and torch.equal(q, wq) and torch.equal(s, ws)


def test_forward_in_place():
    p, _, _ = problem(37, 2048, 1)
    kw = dict(w_post=p["w_post"], w_pre=p["w_pre"], gate=p["gate"], scale=0.5)
    res, z = bs.block_norm(p["x"], p["residual"], **kw)
    inplace = p["residual"].clone()
    res2, z2 = bs.block_norm(p["x"], inplace, res_out=inplace, **kw)
    assert res2 is inplace and torch.equal(res, res2) and torch.equal(z, z2)
    inplace = p["x"].clone()
    res3, z3 = bs.block_norm(inplace, p["residual"], res_out=inplace, **kw)
    assert torch.equal(res, res3) and torch.equal(z, z3)


def test_forward_degenerate_rows():
    p, _, _ = problem(6, 264, 1)
    p["x"][0] = 0.0
    p["residual"][0] = 0.0           # a zero row: rstd = 1 / sqrt(eps)
    p["x"][1] *= 1e30                # squares beyond binary32
    p["residual"][1] *= 1e30
    p["x"][2] *= 1e-30               # squares below it
    p["x"][3, 7] = float("inf")
    p["residual"][4, 9] = float("nan")
    kw = dict(w_post=p["w_post"], w_pre=p["w_pre"], gate=p["gate"], scale=1.0, eps=EPS)
    res, z = bs.block_norm(p["x"], p["residual"], **kw)
    wres, wz = R.norm_steps(p["x"], p["residual"], p["w_post"], p["w_pre"], p["gate"], 1.0, EPS)
    same = lambda a, b: torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(1.0), b.nan_to_num(1.0))  # noqa: E731
    assert same(res, wres) and same(z, wz)
    _, q, s = bs.block_norm(p["x"], p["residual"], fmt="int8", **kw)
    assert s[4].isnan() and (q[4] == 0).all() and torch.equal(q[:3], bs.int8_quantize(z[:3])[0])


def reference_backward(dres, dz, p, res, scale):
    """64-bit gradients by autograd of the 64-bit function, and bounds of the binary32 evaluation."""
    H = p["residual"].shape[1]
    leaf = lambda t: None if t is None else t.double().detach().requires_grad_()  # noqa: E731
    d = torch.zeros_like(p["residual"], dtype=torch.float64) if dres is None else dres.double()
    mag = d.abs()
    out = {}
    if dz is not None:
        r, w = leaf(res), leaf(p["w_pre"])
        z = r / torch.sqrt((r * r).mean(dim=1, keepdim=True) + EPS) * w
        gr, gw = torch.autograd.grad(z, (r, w), dz.double())
        zh, rs = (z / w).detach(), R.rstd(res, EPS)
        gz = (dz.double() * w).detach()
        mag = mag + rs * (gz.abs() + zh.abs() * (gz * zh).abs().mean(dim=1, keepdim=True))
        out["dw_pre"] = (gw, (dz.double() * zh).abs().sum(0))
        d = d + gr
    out["dres"] = (d, mag)
    if p["x"] is not None:
        x, w, gate = leaf(p["x"]), leaf(p["w_post"]), leaf(p["gate"])
        y = R.norm64(x, torch.zeros_like(x), w, gate, scale, EPS)
        wanted = [t for t in (x, w, gate) if t is not None]
        grads = dict(zip([n for n, t in (("dx", x), ("dw_post", w), ("dgate", gate)) if t is not None],
                         torch.autograd.grad(y, wanted, d)))
        T = x.shape[0]
        g = torch.full_like(x, scale)
        if gate is not None:
            rows = gate.detach().reshape(-1, H)
            g = rows.repeat_interleave(T // rows.shape[0], dim=0) * scale
        xs = R.rstd(p["x"], EPS) if w is not None else torch.ones((T, 1), device=DEV, dtype=torch.float64)
        xh = (x * xs).detach()
        gx = (mag * g.abs() * (1 if w is None else w.abs())).detach()
        if w is None:
            out["dx"] = (grads["dx"], gx)
        else:
            out["dx"] = (grads["dx"], xs * (gx + xh.abs() * (gx * xh.abs()).mean(dim=1, keepdim=True)))
            out["dw_post"] = (grads["dw_post"], (mag * g.abs() * xh.abs()).sum(0))
        if gate is not None:
            n = xh if w is None else xh * w.detach()
            rows = p["gate"].reshape(-1, H).shape[0]
            m = (mag * abs(scale) * n.abs()).view(rows, T // rows, H).sum(1)
            out["dgate"] = (grads["dgate"], m.view(grads["dgate"].shape))
    return out


@pytest.mark.parametrize("T,H,groups", [s for s in SHAPES] + [(515, 2056, 1), (1030, 512, 5), (4100, 64, 2), (64, 8192, -1),
                                                             (40, 16384, 8)])
@pytest.mark.parametrize("parts", ["all", "no_post", "no_pre", "pre_only", "no_dres"])
def test_backward(T, H, groups, parts):
    p, dres, dz = problem(T, H, groups, seed=5)
    if parts == "no_post":
        p["w_post"] = None
    if parts == "no_pre":
        p["w_pre"], dz = None, None
    if parts == "pre_only":
        p["x"] = p["w_post"] = p["gate"] = None
    if parts == "no_dres":
        dres = None
    kw = dict(w_post=p["w_post"], w_pre=p["w_pre"], gate=p["gate"], scale=0.3, eps=EPS)
    fwd = bs.block_norm(p["x"], p["residual"], **kw)
    res = fwd[0] if p["w_pre"] is not None else fwd
    names = ("dx", "dres", "dw_post", "dw_pre", "dgate")
    got = dict(zip(names, bs.block_norm_backward(dres, dz, p["x"], res if dz is not None else None, **kw)))
    want = reference_backward(dres, dz, p, res, 0.3)
    assert {n for n in names if got[n] is not None} == set(want)
    for n, (ref, mag) in want.items():
        # about twenty binary32 roundings of terms no larger than mag per element, a row's mean sums in 64 bits of
        # 8-term binary32 dots; the vectors sum T such terms in binary32
        if n in ("dx", "dres"):
            R.check(got[n], ref, 64 * R.F32 * mag, f"{n} {parts}")
        else:
            assert got[n].dtype == torch.float32
            err = (got[n].double() - ref).abs()
            bound = (64 + T) * R.F32 * mag + 1e-40
            assert (err <= bound).all(), (n, (err / bound).max().item())
    again = dict(zip(names, bs.block_norm_backward(dres, dz, p["x"], res if dz is not None else None, **kw)))
    assert all(got[n] is None or torch.equal(got[n], again[n]) for n in names)


@pytest.mark.parametrize("T,H", [(6000, 8192), (9000, 2048)])
@pytest.mark.parametrize("parts", ["no_post", "pre_only"])
def test_backward_long_strips_without_post_norm(T, H, parts):
    """Many rows per workgroup with one reduction each: every row's sums are its own, the first time and again."""
    p, dres, dz = problem(T, H, 1, seed=11)
    p["w_post"] = None
    if parts == "pre_only":
        p["x"] = p["gate"] = None
    kw = dict(w_post=None, w_pre=p["w_pre"], gate=p["gate"], scale=0.3, eps=EPS)
    res, _ = bs.block_norm(p["x"], p["residual"], **kw)
    got = bs.block_norm_backward(dres, dz, p["x"], res, **kw)
    ref, mag = reference_backward(dres, dz, p, res, 0.3)["dres"]
    R.check(got[1], ref, 64 * R.F32 * mag, parts)
    for _ in range(3):
        again = bs.block_norm_backward(dres, dz, p["x"], res, **kw)
        assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


def test_backward_against_differences():
    """L = sum(dres res) + sum(dz z) as a 64-bit function of every input (res unrounded), central differences along
    random directions.  The kernel takes the gradient at the stored (rounded) res: 2^-8 of it, averaged."""
    T, H = 24, 96
    p, dres, dz = problem(T, H, 3, seed=9)
    kw = dict(w_post=p["w_post"], w_pre=p["w_pre"], gate=p["gate"], scale=0.7, eps=EPS)
    res, _ = bs.block_norm(p["x"], p["residual"], **kw)
    dx, dr, dwp, dwn, dg = bs.block_norm_backward(dres, dz, p["x"], res, **kw)

    def loss(q):
        r = R.norm64(q["x"], q["residual"], q["w_post"], q["gate"], 0.7, EPS)
        z = r / torch.sqrt((r * r).mean(dim=1, keepdim=True) + EPS) * q["w_pre"]
        return (r * dres.double()).sum() + (z * dz.double()).sum()

    t = 1e-5
    base = {k: v.double() for k, v in p.items()}
    for name, grad in (("x", dx), ("residual", dr), ("w_post", dwp), ("w_pre", dwn), ("gate", dg)):
        E = torch.randn(base[name].shape, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV, dtype=torch.float64)
        diff = (loss({**base, name: base[name] + t * E}) - loss({**base, name: base[name] - t * E})) / (2 * t)
        got = (grad.double() * E).sum()
        assert (got - diff).abs() <= 1e-2 * grad.double().norm(), name


def test_empty():
    p, dres, dz = problem(4, 64, 1)
    kw = dict(w_post=p["w_post"], w_pre=p["w_pre"], gate=p["gate"])
    res, z = bs.block_norm(p["x"][:0], p["residual"][:0], **kw)
    assert res.shape == z.shape == (0, 64)
    dx, dr, dwp, dwn, dg = bs.block_norm_backward(dres[:0], dz[:0], p["x"][:0], res, **kw)
    assert dx.shape == dr.shape == (0, 64) and (dwp == 0).all() and (dwn == 0).all() and (dg == 0).all()


def additions(T, H, groups):
    """The longest chain of additions behind a vector gradient: the rows of a strip one by one, then the strips'
    partials (every 64th in one thread, the 64 threads' in two steps and fifteen more additions)."""
    chunks, nt = H // 8, 64
    while nt < min(1024, chunks):
        nt *= 2
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    want = min(min(1024, cus * (1024 // nt)), max(min(T, cus), T // 4))
    if groups >= want:
        per = -(-groups // want)
        strips, rows = -(-groups // per), per * (T // groups)
    else:
        parts = min(T // groups, -(-want // groups))
        strips, rows = groups * parts, -(-(T // groups) // parts)
    return rows + -(-strips // 64) + 17


@pytest.mark.parametrize("T,H,groups", [(8192, 4096, 1), (1500, 8192, 1), (1100, 16384, 2), (2050, 8200, 1), (6000, 7168, 3),
                                        (9000, 2048, -1), (9000, 264, 3000), (20000, 512, 5)])
@pytest.mark.parametrize("parts", ["all", "no_post", "no_pre", "pre_only", "no_dres", "no_gate"])
def test_backward_many_rows_per_strip(T, H, groups, parts):
    """Every output against 64 bits where a workgroup walks several rows, at every width of the kernels.  A vector's
    gradient: its terms' 64 roundings, and one for every addition that a term passes through."""
    p, dres, dz = problem(T, H, groups, seed=13)
    if parts == "no_post":
        p["w_post"] = None
    if parts == "no_pre":
        p["w_pre"], dz = None, None
    if parts == "pre_only":
        p["x"] = p["w_post"] = p["gate"] = None
    if parts == "no_dres":
        dres = None
    if parts == "no_gate":
        p["gate"] = None
    kw = dict(w_post=p["w_post"], w_pre=p["w_pre"], gate=p["gate"], scale=0.3, eps=EPS)
    fwd = bs.block_norm(p["x"], p["residual"], **kw)
    res = fwd[0] if p["w_pre"] is not None else fwd
    names = ("dx", "dres", "dw_post", "dw_pre", "dgate")
    got = dict(zip(names, bs.block_norm_backward(dres, dz, p["x"], res if dz is not None else None, **kw)))
    want = reference_backward(dres, dz, p, res, 0.3)
    assert {n for n in names if got[n] is not None} == set(want)
    n_add = additions(T, H, 1 if p["gate"] is None else p["gate"].reshape(-1, H).shape[0])
    assert T <= 1024 or n_add < T // 2  # a bound far below one by the number of rows
    for n, (ref, mag) in want.items():
        if n in ("dx", "dres"):
            R.check(got[n], ref, 64 * R.F32 * mag, f"{n} {parts}")
        else:
            err, bound = (got[n].double() - ref).abs(), (64 + n_add) * R.F32 * mag + 1e-40
            assert (err <= bound).all(), (n, (err / bound).max().item())
