"""GPU: the block operators as they are used together: a feed-forward block served at 8 bits, one trained in bf16,
on other streams, and captured into graphs that are replayed with the program's eager work in between."""
import ctypes

import pytest
import torch

import block_scaled_fp4_e2m1_amd as bs
import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6


class Block:
    """norm -> 8-bit quantise -> 8-bit gated -> 8-bit linear -> norm, gate, residual, next norm."""

    def __init__(self, T, H, I, seed=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        bf = lambda *s, std=1.0, mean=0.0: (torch.randn(s, generator=g, device=DEV) * std + mean).to(torch.bfloat16)  # noqa: E731
        self.residual, self.w_in, self.w_post, self.w_next = bf(T, H, std=2.0), bf(H, std=0.1, mean=1), bf(H, mean=1), bf(H, mean=1)
        self.gate = bf(H)
        self.w13, self.w2 = bf(2 * I, H, std=H ** -0.5), bf(H, I, std=I ** -0.5)
        self.q13, self.s13 = bs.int8_quantize(self.w13)   # a weight row is an output channel
        self.q2, self.s2 = bs.int8_quantize(self.w2)

    def serve(self):
        _, q, s = bs.block_norm(None, self.residual, w_pre=self.w_in, fmt="int8")
        h = bs.int8_gated_ffn(q, s, self.q13, self.s13)
        y = bs.int8_quantize_gemm(h, self.q2, self.s2)
        res, z = bs.block_norm(y, self.residual, w_post=self.w_post, w_pre=self.w_next, gate=self.gate, scale=0.5)
        return q, s, h, y, res, z

    def train(self, dres, dz):
        _, z0 = bs.block_norm(None, self.residual, w_pre=self.w_in)
        h, gu = bs.gated_ffn(z0, self.w13, save_gate_up=True)
        res, z = bs.block_norm(h, self.residual, w_post=self.w_post, w_pre=self.w_next, gate=self.gate, scale=0.5)
        dh, dr, dwp, dwn, dg = bs.block_norm_backward(dres, dz, h, res, w_post=self.w_post, w_pre=self.w_next,
                                                      gate=self.gate, scale=0.5)
        dz0, dw13 = bs.gated_ffn_backward(dh, z0, self.w13, gu)
        _, dr2, _, dwi, _ = bs.block_norm_backward(dr, dz0, None, self.residual, w_pre=self.w_in)
        return h, res, z, dw13, dr2, dwp, dwn, dg, dwi


@pytest.mark.parametrize("T,H,I", [(1, 512, 272), (37, 1024, 784), (300, 512, 1536)])
def test_serving_chain(T, H, I):
    """Each stage against 64 bits, given the stage before it."""
    b = Block(T, H, I)
    q, s, h, y, res, z = b.serve()
    zin = R.norm_steps(None, b.residual, None, b.w_in, None, 1.0, EPS)[1]
    wq, ws = R.int8_rows(zin)
    assert torch.equal(q, wq) and torch.equal(s, ws)
    y13 = R.int8_product(q, s, b.q13, b.s13)
    G, U = y13[:, :I], y13[:, I:]
    R.gated_check(h, G, U, 3.1 * R.F32 * G.abs(), 3.1 * R.F32 * U.abs(), "silu", "h")
    hq, hs = R.int8_rows(h)
    ref = R.int8_product(hq, hs, b.q2, b.s2)
    R.check(y, ref, 3.1 * R.F32 * ref.abs(), "y")
    wres, wz = R.norm_steps(y, b.residual, b.w_post, b.w_next, b.gate, 0.5, EPS)
    assert torch.equal(res, wres) and torch.equal(z, wz)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_norm_feeds_the_fp4_quantiser(fmt):
    b = Block(19, 512, 64)
    _, z = bs.block_norm(None, b.residual, w_pre=b.w_in)
    wz = R.norm_steps(None, b.residual, None, b.w_in, None, 1.0, EPS)[1]
    gs = bs.global_scale(z) if fmt == "nvfp4" else None
    for a, c in zip(bs.quantize(z, fmt, gs=gs), bs.quantize(wz.contiguous(), fmt, gs=gs)):
        assert torch.equal(a, c)


@pytest.mark.parametrize("device", [0, "cuda", "cuda:0", torch.device("cuda"), torch.device("cuda:0")], ids=repr)
def test_current_stream_of_any_device_form(device):
    """The binding's stream handle, for whatever names a device."""
    from block_scaled_fp4_e2m1_amd import binding
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert binding._stream(device).value == side.cuda_stream
    assert (binding._stream(device).value or 0) == torch.cuda.current_stream().cuda_stream


def test_other_streams_and_two_at_once():
    b1, b2 = Block(64, 1024, 512, 1), Block(130, 512, 784, 2)
    want1, want2 = b1.serve(), b2.serve()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got1, got2 = [], []
    for _ in range(3):
        with torch.cuda.stream(s1):
            got1.append(b1.serve())
        with torch.cuda.stream(s2):
            got2.append(b2.serve())
    torch.cuda.synchronize()
    assert all(torch.equal(a, w) for g in got1 for a, w in zip(g, want1))
    assert all(torch.equal(a, w) for g in got2 for a, w in zip(g, want2))


def _capture(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fn()
    return g, out


@pytest.mark.parametrize("T,H,I", [(1, 1024, 1024), (70, 512, 512)])
def test_graphs(T, H, I):
    """A serving and a training pass, each captured once; replays between eager passes on new inputs give the eager
    bits, also with both graphs alive."""
    b = Block(T, H, I, 3)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    dres, dz = torch.zeros_like(b.residual), torch.zeros_like(b.residual)
    gs, out_s = _capture(b.serve)
    gt, out_t = _capture(lambda: b.train(dres, dz))
    for _ in range(3):
        for t in (b.residual, dres, dz):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV).to(torch.bfloat16))
        want_s, want_t = b.serve(), b.train(dres, dz)
        torch.cuda.synchronize()
        gt.replay()
        gs.replay()
        torch.cuda.synchronize()
        for a, w in zip((*out_s, *out_t), (*want_s, *want_t)):
            assert torch.equal(a, w)


def test_overlapping_outputs_are_refused():
    x = torch.randn((70, 64), device=DEV).to(torch.bfloat16)
    W = torch.randn((128, 64), device=DEV).to(torch.bfloat16)
    q, s = bs.int8_quantize(W[:64].contiguous())
    before = x.clone()
    for call in (lambda: bs.gated_ffn(x, W, out=x), lambda: bs.int8_quantize_gemm(x, q, s, out=x),
                 lambda: bs.block_norm(x[:-1], W[:69], res_out=x[1:])):
        with pytest.raises(bs.Bsfp4Error, match="overlaps"):
            call()
    torch.cuda.synchronize()
    assert torch.equal(x, before)


def test_training_chain_against_differences():
    """The whole trained block's gradient with respect to its weight and its input, along random directions, against
    central differences of the 64-bit block (no roundings in between).  Every stage's bf16 rounding enters the
    gradient with random signs: 2 % of its norm along a direction of unit elements bounds their sum generously (six
    roundings of 2^-8 at most per term)."""
    T, H, I = 40, 128, 128
    b = Block(T, H, I, 7)
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    dres, dz = (torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    out = b.train(dres, dz)
    dw13, dr = out[3].double(), out[4].double()

    def loss(res0, w13):
        n = lambda v, w: v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS) * w.double()  # noqa: E731
        y = n(res0, b.w_in) @ w13.t()
        h = R.act("silu", y[:, :I])[0] * y[:, I:]
        r = res0 + 0.5 * b.gate.double() * n(h, b.w_post)
        return (r * dres.double()).sum() + (n(r, b.w_next) * dz.double()).sum()

    t = 1e-5
    r0, w0 = b.residual.double(), b.w13.double()
    for which, grad in ((0, dr), (1, dw13)):
        E = torch.randn(grad.shape, generator=g, device=DEV, dtype=torch.float64)
        args = lambda sgn: (r0 + sgn * t * E, w0) if which == 0 else (r0, w0 + sgn * t * E)  # noqa: E731
        diff = (loss(*args(1)) - loss(*args(-1))) / (2 * t)
        assert ((grad * E).sum() - diff).abs() <= 2e-2 * grad.norm()


def test_aliased_python_outputs_are_refused():
    """out= and q= that share memory with an operand other workgroups still read."""
    K = 128
    A = torch.randint(-128, 128, (70, K), device=DEV, dtype=torch.int8)
    W = torch.randint(-128, 128, (128, K), device=DEV, dtype=torch.int8)
    SA, SW = torch.ones(70, device=DEV), torch.ones(128, device=DEV)
    x = torch.randn((70, 64), device=DEV).to(torch.bfloat16)
    before = A.clone(), x.clone()
    over = A.view(torch.bfloat16)                             # [70, 64] on A's own bytes
    for call in (lambda: bs.int8_gemm(A, SA, W[:64], SW[:64], out=over), lambda: bs.int8_gated_ffn(A, SA, W, SW, out=over),
                 lambda: bs.int8_quantize(x, q=x.view(torch.int8).view(-1)[:70 * 64].view(70, 64)),
                 lambda: bs.int8_quantize(x, s=x.view(-1).view(torch.float32)[:70])):
        with pytest.raises(bs.Bsfp4Error, match="overlaps"):
            call()
    torch.cuda.synchronize()
    assert torch.equal(A, before[0]) and torch.equal(x, before[1])


@pytest.mark.parametrize("T,H", [(300, 512), (700, 4096), (90, 8712)])
def test_gradients_in_place(T, H):
    """Row gradients of the norm over their own inputs, and dx of the gated product over an x that is not read."""
    from block_scaled_fp4_e2m1_amd import binding
    g = torch.Generator(device=DEV)
    g.manual_seed(T + H)
    x, residual, dres, dz = (torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16) for _ in range(4))
    wp, wn, gate = (torch.randn(H, generator=g, device=DEV).to(torch.bfloat16) for _ in range(3))
    kw = dict(w_post=wp, w_pre=wn, gate=gate, scale=0.5)
    res, z = bs.block_norm(x, residual, **kw)
    want = bs.block_norm_backward(dres, dz, x, res, **kw)
    lib = binding.load()
    n = lib.bsfp4_block_norm_backward_workspace_size(T, H, 1)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    for ox, od in (("x", "res_out"), ("dz", "dres_out"), ("res_out", "x"), ("dres_out", "dz")):
        t = dict(x=x.clone(), res_out=res.clone(), dres_out=dres.clone(), dz=dz.clone())
        vecs = [torch.empty(H, device=DEV) for _ in range(3)]
        a = binding.BlockNormArgs(scale=0.5, eps=1e-6, T=T, H=H, groups=1, w_post=wp.data_ptr(), w_pre=wn.data_ptr(),
                                  gate=gate.data_ptr(), dx=t[ox].data_ptr(), dres=t[od].data_ptr(),
                                  **{k: v.data_ptr() for k, v in t.items()},
                                  **dict(zip(("dw_post", "dw_pre", "dgate"), (v.data_ptr() for v in vecs))))
        assert lib.bsfp4_block_norm_backward(ctypes.byref(a), ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == 0
        for got, w in zip((t[ox], t[od], *vecs), want):
            assert torch.equal(got, w)
    a = binding.BlockNormArgs(scale=0.5, eps=1e-6, T=T, H=H, groups=1, w_pre=wn.data_ptr(), x=x.data_ptr(),
                              residual=residual.data_ptr())
    wres, wz = bs.block_norm(x, residual, w_pre=wn, scale=0.5)
    xi, ri = x.clone(), residual.clone()
    a.x, a.residual, a.res_out, a.z = xi.data_ptr(), ri.data_ptr(), xi.data_ptr(), ri.data_ptr()
    assert lib.bsfp4_block_norm(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(xi, wres) and torch.equal(ri, wz)


def test_gated_gradient_over_an_unread_operand():
    from block_scaled_fp4_e2m1_amd import binding
    M, H, I = 333, 264, 136
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x, dh, W = (torch.randn(s, generator=g, device=DEV).to(torch.bfloat16) for s in ((M, H), (M, I), (2 * I, H)))
    _, gu = bs.gated_ffn(x, W, save_gate_up=True)
    dx, dW = bs.gated_ffn_backward(dh, x, W, gu)
    lib = binding.load()
    n = lib.bsfp4_gated_ffn_backward_workspace_size(M, I, H)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)

    def call(dx_at, dW_at, x_at, W_at):
        st = torch.cuda.current_stream().cuda_stream
        p = [None if t is None else t.data_ptr() for t in (dh, x_at, W_at, gu)]
        assert lib.bsfp4_gated_ffn_backward(*p, 0, *(None if t is None else t.data_ptr() for t in (dx_at, dW_at)), M, I, H,
                                            ws.data_ptr(), n, st) == 0

    xi, Wi = x.clone(), W.clone()
    call(xi, None, xi, W)
    call(None, Wi, x, Wi)
    assert torch.equal(xi, dx) and torch.equal(Wi, dW)
