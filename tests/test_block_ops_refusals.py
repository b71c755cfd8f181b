"""CPU: what the 8-bit, gated feed-forward and block-norm entry points refuse, in the binding (extents, types: meta
tensors, nothing reaches the library) and in the C ABI (no kernel is launched: every call fails validation)."""
import ctypes

import pytest
import torch

import block_scaled_fp4_e2m1_amd as bs
from block_scaled_fp4_e2m1_amd import binding

I8, BF16, F32 = torch.int8, torch.bfloat16, torch.float32
OK, INVALID, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
FAKE = 0x100000


def m(*shape, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="meta")


def reaches_device_check(fn, *a, **kw):
    with pytest.raises(ValueError, match="must be a device tensor"):
        fn(*a, **kw)


def refused(match, fn, *a, error=ValueError, **kw):
    with pytest.raises(error, match=match):
        fn(*a, **kw)


def test_int8_quantize():
    reaches_device_check(bs.int8_quantize, m(4, 64))
    reaches_device_check(bs.int8_quantize, m(4, 64), q=m(4, 64, dtype=I8), s=m(4, dtype=F32))
    refused("multiple of 8", bs.int8_quantize, m(4, 60))
    refused("2-D", bs.int8_quantize, m(64))
    refused("contiguous", bs.int8_quantize, m(64, 4).t())
    refused("bfloat16", bs.int8_quantize, m(4, 64, dtype=F32), error=TypeError)
    refused("q must have shape", bs.int8_quantize, m(4, 64), q=m(4, 56, dtype=I8))
    refused("s must have shape", bs.int8_quantize, m(4, 64), s=m(5, dtype=F32))


def test_int8_gemm():
    A, SA, B, SB = m(4, 64, dtype=I8), m(4, dtype=F32), m(24, 64, dtype=I8), m(24, dtype=F32)
    f = bs.int8_gemm
    reaches_device_check(f, A, SA, B, SB)
    reaches_device_check(f, A, SA, B, SB, bias=m(24), out=m(4, 24))
    refused("K=64 but B has K=80", f, A, SA, m(24, 80, dtype=I8), SB)
    refused("multiple of 16", f, m(4, 72, dtype=I8), SA, m(24, 72, dtype=I8), SB)
    refused("N=20", f, A, SA, m(20, 64, dtype=I8), m(20, dtype=F32))
    refused("SA must have", f, A, m(5, dtype=F32), B, SB)
    refused("SB must have", f, A, SA, B, m(23, dtype=F32))
    refused("bias must have", f, A, SA, B, SB, bias=m(23))
    refused("out must have", f, A, SA, B, SB, out=m(4, 16))
    refused("bfloat16", f, A, SA, B, SB, bias=m(24, dtype=F32), error=TypeError)
    refused("int8", f, m(4, 64), SA, B, SB, error=TypeError)
    g = bs.int8_quantize_gemm
    reaches_device_check(g, m(4, 64), B, SB)
    refused("K=80 but B has K=64", g, m(4, 80), B, SB)
    refused("out must have", g, m(4, 64), B, SB, out=m(5, 24))


def test_gated():
    A, SA, W, SW = m(4, 64, dtype=I8), m(4, dtype=F32), m(32, 64, dtype=I8), m(32, dtype=F32)
    reaches_device_check(bs.int8_gated_ffn, A, SA, W, SW, act="gelu")
    refused("unknown activation", bs.int8_gated_ffn, A, SA, W, SW, act="relu")
    refused("as many up rows", bs.int8_gated_ffn, A, SA, m(33, 64, dtype=I8), m(33, dtype=F32))
    refused("I=12", bs.int8_gated_ffn, A, SA, m(24, 64, dtype=I8), m(24, dtype=F32))
    refused("SW13 must have", bs.int8_gated_ffn, A, SA, W, m(16, dtype=F32))
    refused("out must have", bs.int8_gated_ffn, A, SA, W, SW, out=m(4, 32))
    x, W = m(4, 64), m(32, 64)
    reaches_device_check(bs.gated_ffn, x, W, act="gelu_tanh", save_gate_up=True)
    refused("W13 has H=56", bs.gated_ffn, x, m(32, 56))
    refused("H=60", bs.gated_ffn, m(4, 60), m(32, 60))
    refused("unknown activation", bs.gated_ffn, x, W, act=None)
    refused("unknown activation", bs.gated_ffn, x, W, act=["silu"])
    refused("out must have", bs.gated_ffn, x, W, out=m(4, 32))
    dh, gu = m(4, 16), m(4, 32, dtype=F32)
    reaches_device_check(bs.gated_ffn_backward, dh, x, W, gu)
    refused("dh must have", bs.gated_ffn_backward, m(4, 32), x, W, gu)
    refused("gate_up must have", bs.gated_ffn_backward, dh, x, W, m(4, 16, dtype=F32))
    refused("float32", bs.gated_ffn_backward, dh, x, W, m(4, 32), error=TypeError)
    refused("contiguous", bs.gated_ffn_backward, dh, x, W, m(32, 4, dtype=F32).t())


def test_block_norm():
    x, r, w = m(6, 64), m(6, 64), m(64)
    f = bs.block_norm
    reaches_device_check(f, x, r, w_post=w, w_pre=w, gate=m(3, 64))
    reaches_device_check(f, None, r, w_pre=w, fmt="int8")
    reaches_device_check(f, x, r, gate=w)
    refused("x must have", f, m(6, 56), r)
    refused("H=60", f, None, m(6, 60), w_pre=m(60))
    refused("w_post must have", f, x, r, w_post=m(56))
    refused("w_pre must have", f, x, r, w_pre=m(1, 64))
    refused("gate must have", f, x, r, gate=m(3, 56))
    refused("gate must have", f, x, r, gate=m(1, 3, 64))
    refused("not a multiple of the 4", f, x, r, gate=m(4, 64))
    refused("not a multiple of the 0", f, x, r, gate=m(0, 64))
    refused("without x", f, None, r, w_post=w, w_pre=w)
    refused("without x", f, None, r, w_pre=w, gate=w)
    refused("nothing is written", f, None, r, w_pre=w, res_out=m(6, 64))
    refused("neither x nor w_pre", f, None, r)
    refused("unknown output format", f, x, r, w_pre=w, fmt="nvfp4")
    refused("needs w_pre", f, x, r, fmt="int8")
    refused("eps", f, x, r, eps=0.0)
    refused("eps", f, x, r, eps=float("nan"))
    refused("bfloat16", f, x, r, w_pre=m(64, dtype=F32), error=TypeError)
    b = bs.block_norm_backward
    reaches_device_check(b, r, r, x, r, w_post=w, w_pre=w, gate=w)
    reaches_device_check(b, None, r, None, r, w_pre=w)
    refused("w_pre needs", b, r, None, x, r, w_pre=w)
    refused("w_pre needs", b, r, r, x, None, w_pre=w)
    refused("dz without", b, r, r, x, r)
    refused("dres is needed", b, None, None, x, r)
    refused("dz must have", b, r, m(5, 64), x, r, w_pre=w)


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def err(lib):
    return lib.bsfp4_last_error().decode()


def test_abi_int8(lib):
    f = lib.bsfp4_int8_quantize
    assert f(FAKE, 2, 20, FAKE, FAKE, None) == SHAPE and "multiple of 8" in err(lib)
    assert f(FAKE, -1, 16, FAKE, FAKE, None) == SHAPE
    assert f(None, 2, 16, FAKE, FAKE, None) == INVALID
    assert f(FAKE + 8, 2, 16, FAKE, FAKE, None) == ALIGN
    assert f(FAKE, 2, 16, FAKE, FAKE + 2, None) == ALIGN
    assert f(None, 0, 16, None, None, None) == OK
    assert f(FAKE, 1 << 26, 16, FAKE, FAKE, None) == SHAPE and f(FAKE, 1 << 25, 256, FAKE, FAKE, None) == SHAPE
    g = lib.bsfp4_int8_gemm

    def call(A=FAKE, sa=FAKE, B=FAKE, sb=FAKE, bias=None, D=FAKE, M=2, N=64, K=64, ws=None, n=0):
        return g(A, sa, B, sb, bias, D, M, N, K, ws, n, None)

    assert call(N=60) == SHAPE and "multiple of 8" in err(lib)
    assert call(K=72) == SHAPE and "multiple of 16" in err(lib)
    assert call(K=131072) == SHAPE and "131056" in err(lib)
    assert call(M=1 << 31) == SHAPE
    assert call(M=(1 << 31) - 1, N=1 << 20) == SHAPE and "2^40" in err(lib)
    assert call(M=(1 << 31) - 1) == SHAPE and "31 bits" in err(lib)  # a tile's rows are counted past M
    assert call(A=None) == INVALID and call(sb=None) == INVALID and call(D=None) == INVALID
    assert call(sb=FAKE + 4) == ALIGN and call(bias=FAKE + 8) == ALIGN
    assert call(M=0, A=None, sa=None, D=None) == OK
    need = lib.bsfp4_int8_quantize_gemm_workspace_size(100, 64, 64)
    assert need >= 100 * 64 + 400
    h = lib.bsfp4_int8_quantize_gemm
    assert h(FAKE, FAKE, FAKE, None, FAKE, 100, 64, 64, FAKE, need - 1, None) == WORKSPACE
    assert h(FAKE, FAKE, FAKE, None, FAKE, 100, 64, 64, None, need, None) == WORKSPACE
    assert h(FAKE, FAKE, FAKE, None, FAKE, 100, 64, 64, FAKE + 4, need, None) == ALIGN
    k = lib.bsfp4_int8_gated_ffn
    assert k(FAKE, FAKE, FAKE, FAKE, 3, FAKE, 2, 64, 64, None, 0, None) == INVALID and "activation" in err(lib)
    assert k(FAKE, FAKE, FAKE, FAKE, 0, FAKE, 2, 60, 64, None, 0, None) == SHAPE


def test_abi_gated(lib):
    f = lib.bsfp4_gated_ffn
    assert f(FAKE, FAKE, -1, FAKE, None, 2, 64, 64, None, 0, None) == INVALID
    assert f(FAKE, FAKE, 0, FAKE, None, 2, 64, 60, None, 0, None) == SHAPE
    assert f(FAKE, FAKE, 0, FAKE, None, 2, 64, 1 << 22, None, 0, None) == SHAPE and "2^22" in err(lib)
    assert f(FAKE, FAKE, 0, FAKE, None, 2, 1 << 21, 64, None, 0, None) == SHAPE
    assert f(FAKE, None, 0, FAKE, None, 2, 64, 64, None, 0, None) == INVALID
    assert f(FAKE, FAKE, 0, FAKE, FAKE + 2, 2, 64, 64, None, 0, None) == ALIGN
    b = lib.bsfp4_gated_ffn_backward
    need = lib.bsfp4_gated_ffn_backward_workspace_size(100, 64, 64)
    assert need >= 100 * 128 * 2
    assert b(FAKE, FAKE, FAKE, FAKE, 0, FAKE, FAKE, 100, 64, 64, FAKE, need - 1, None) == WORKSPACE
    assert b(FAKE, FAKE, FAKE, FAKE, 0, None, None, 100, 64, 64, FAKE, need, None) == INVALID
    assert b(FAKE, FAKE, FAKE, FAKE, 0, FAKE + 8, FAKE, 100, 64, 64, FAKE, need, None) == ALIGN
    assert b(FAKE, None, FAKE, FAKE, 0, FAKE, FAKE, 100, 64, 64, FAKE, need, None) == INVALID
    assert b(None, None, FAKE, None, 0, FAKE, None, 0, 64, 64, FAKE, need, None) == OK


def test_abi_block_norm(lib):
    def call(back=False, ws=FAKE, n=1 << 30, **kw):
        a = binding.BlockNormArgs(scale=1.0, eps=1e-6, T=4, H=64, groups=1, residual=FAKE)
        for k, v in kw.items():
            setattr(a, k, v)
        if back:
            return lib.bsfp4_block_norm_backward(ctypes.byref(a), ws, n, None)
        return lib.bsfp4_block_norm(ctypes.byref(a), None)

    assert lib.bsfp4_block_norm(None, None) == INVALID
    assert call(H=60) == SHAPE and call(H=16392) == SHAPE and call(T=-1) == SHAPE and call(groups=0) == SHAPE
    assert call(T=1 << 26) == SHAPE and call(T=1 << 20, H=8192) == SHAPE and "2^33" in err(lib)
    assert call(x=FAKE, res_out=FAKE, gate=FAKE, groups=3) == SHAPE
    assert call(x=FAKE, res_out=FAKE, groups=2) == SHAPE and "without a gate" in err(lib)
    assert call(x=FAKE, res_out=FAKE, eps=0.0) == INVALID
    assert call() == INVALID                                    # neither x nor w_pre
    assert call(w_post=FAKE, w_pre=FAKE, z=FAKE) == INVALID     # w_post without x
    assert call(x=FAKE) == INVALID                              # no res_out
    assert call(w_pre=FAKE) == INVALID                          # no z
    assert call(w_pre=FAKE, z=FAKE, q=FAKE, s=FAKE) == INVALID
    assert call(w_pre=FAKE, q=FAKE) == INVALID
    assert call(x=FAKE, res_out=FAKE, z=FAKE) == INVALID        # z without w_pre
    assert call(w_pre=FAKE + 8, z=FAKE) == ALIGN and "w_pre" in err(lib)
    assert call(w_pre=FAKE, z=FAKE, residual=None) == INVALID
    assert call(T=0, residual=None, w_pre=FAKE) == OK
    b = dict(back=True, x=FAKE, w_post=FAKE, w_pre=FAKE, res_out=FAKE, dz=FAKE, dx=FAKE, dres=FAKE, dw_post=FAKE,
             dw_pre=FAKE)
    for missing in ("res_out", "dz", "dx", "dres", "dw_post", "dw_pre"):
        assert call(**{**b, missing: None}) == INVALID, missing
    assert call(**b, gate=FAKE) == INVALID and "dgate" in err(lib)
    assert call(**b, n=16) == WORKSPACE


def test_abi_overlapping_outputs(lib):
    """Outputs that share bytes with an input other workgroups still read."""
    far = FAKE + (1 << 32)
    f = lib.bsfp4_int8_quantize_gemm
    for D in (far, far + 2 * 64 - 16, far - 2 * 64 + 16):
        assert f(far, FAKE, FAKE, None, D, 1, 64, 64, None, 0, None) == INVALID and "overlaps" in err(lib)
    f = lib.bsfp4_gated_ffn
    for x, W, h in ((far, FAKE, far), (FAKE, far, far + 2 * 32 * 64 - 16), (far, FAKE, far + 4 * 64 * 2 - 16)):
        assert f(x, W, 0, h, None, 4, 16, 64, FAKE, 1 << 30, None) == INVALID and "overlaps" in err(lib)
    for res_out in (far + 128, far - 128):
        for kw in (dict(x=far, residual=FAKE), dict(x=FAKE, residual=far)):
            a = binding.BlockNormArgs(scale=1.0, eps=1e-6, T=4, H=64, groups=1, res_out=res_out, **kw)
            assert lib.bsfp4_block_norm(ctypes.byref(a), None) == INVALID and "overlaps" in err(lib)


def test_abi_most_rows(lib):
    """The row kernels launch 256 threads for every four rows, rounded up: fewer than 2^32 in all."""
    most = (1 << 26) - 4
    assert (most + 3) // 4 * 256 < 1 << 32 <= (most + 4) // 4 * 256
    for rows in (most + 1, most + 3):
        assert lib.bsfp4_int8_quantize(FAKE, rows, 8, FAKE, FAKE, None) == SHAPE and "rows" in err(lib)
        a = binding.BlockNormArgs(scale=1.0, eps=1e-6, T=rows, H=8, groups=1, residual=FAKE, w_pre=FAKE, z=FAKE)
        assert lib.bsfp4_block_norm(ctypes.byref(a), None) == SHAPE and "rows" in err(lib)
    # `most` itself passes, to be stopped by what is checked after it
    assert lib.bsfp4_int8_quantize(None, most, 8, FAKE, FAKE, None) == INVALID


# ---- outputs that share memory with an input or with each other, for every pair of every entry point

M_, N_, K_, T_, H_, G_ = 70, 64, 96, 12, 64, 3


def _norm(lib, back):
    def call(p):
        a = binding.BlockNormArgs(scale=1.0, eps=1e-6, T=T_, H=H_, groups=G_)
        for k, v in p.items():
            setattr(a, k, v)
        if back:
            return lib.bsfp4_block_norm_backward(ctypes.byref(a), FAKE, 1 << 30, None)
        return lib.bsfp4_block_norm(ctypes.byref(a), None)
    return call


#: entry -> (outputs, inputs as name -> bytes, the call, pairs that may be the same memory exactly)
def overlap_cases(lib):
    ws = (FAKE, 1 << 30)
    mk, mn, nk, th, v = M_ * K_, M_ * N_, N_ * K_, 2 * T_ * H_, 2 * H_
    norm_in = dict(x=th, residual=th, w_post=v, w_pre=v, gate=G_ * v)
    back_in = dict(x=th, res_out=th, dres_out=th, dz=th, w_post=v, w_pre=v, gate=G_ * v)
    rows = {(o, i) for o in ("dx", "dres") for i in ("x", "res_out", "dres_out", "dz")}
    return {
        "int8_quantize": (dict(q=mk, s=4 * M_), dict(x=2 * mk),
                          lambda p: lib.bsfp4_int8_quantize(p["x"], M_, K_, p["q"], p["s"], None), set()),
        "int8_gemm": (dict(D=2 * mn), dict(A=mk, sa=4 * M_, B=nk, sb=4 * N_, bias=2 * N_),
                      lambda p: lib.bsfp4_int8_gemm(p["A"], p["sa"], p["B"], p["sb"], p["bias"], p["D"], M_, N_, K_, *ws,
                                                    None), set()),
        "int8_quantize_gemm": (dict(D=2 * mn), dict(x=2 * mk, B=nk, sb=4 * N_, bias=2 * N_),
                               lambda p: lib.bsfp4_int8_quantize_gemm(p["x"], p["B"], p["sb"], p["bias"], p["D"], M_, N_,
                                                                      K_, *ws, None), set()),
        "int8_gated_ffn": (dict(h=2 * mn), dict(A=mk, sa=4 * M_, W=2 * nk, sw=8 * N_),
                           lambda p: lib.bsfp4_int8_gated_ffn(p["A"], p["sa"], p["W"], p["sw"], 0, p["h"], M_, N_, K_, *ws,
                                                              None), set()),
        "gated_ffn": (dict(h=2 * mn, gate_up=8 * mn), dict(x=2 * mk, W=4 * nk),
                      lambda p: lib.bsfp4_gated_ffn(p["x"], p["W"], 0, p["h"], p["gate_up"], M_, N_, K_, *ws, None), set()),
        "gated_ffn_backward": (dict(dx=2 * mk, dW=4 * nk), dict(x=2 * mk, W=4 * nk),
                               lambda p: lib.bsfp4_gated_ffn_backward(FAKE, p["x"], p["W"], FAKE, 0, p["dx"], p["dW"], M_,
                                                                      N_, K_, *ws, None), set()),
        "block_norm": (dict(res_out=th, z=th), norm_in, _norm(lib, False),
                       {(o, i) for o in ("res_out", "z") for i in ("x", "residual")}),
        "block_norm int8": (dict(res_out=th, q=th // 2, s=4 * T_), norm_in, _norm(lib, False),
                            {("res_out", "x"), ("res_out", "residual")}),
        "block_norm_backward": (dict(dx=th, dres=th, dw_post=2 * v, dw_pre=2 * v, dgate=2 * G_ * v), back_in,
                                _norm(lib, True), rows),
    }


ENTRIES = ["int8_quantize", "int8_gemm", "int8_quantize_gemm", "int8_gated_ffn", "gated_ffn", "gated_ffn_backward",
           "block_norm", "block_norm int8", "block_norm_backward"]


@pytest.mark.parametrize("entry", ENTRIES)
def test_abi_every_overlap(lib, entry):
    outs, ins, call, same = overlap_cases(lib)[entry]
    every = {**ins, **outs}
    far = {name: (k + 1) << 36 for k, name in enumerate(every)}
    for o in outs:
        for i in every:
            if i == o:
                continue
            # the last 16 bytes, the first, and all of it
            for at in (far[i] + every[i] // 16 * 16 - 16, far[i] - every[o] // 16 * 16 + 16, far[i]):
                if at == far[i] and (o, i) in same:
                    continue
                assert call({**far, o: at}) == INVALID, (o, i, at - far[i])
                assert "overlaps" in err(lib) and o in err(lib) and i in err(lib)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory: only where no kernel can be launched")
@pytest.mark.parametrize("entry", ENTRIES)
def test_abi_memory_side_by_side(lib, entry):
    """Neighbours, and outputs that may be an input itself, are not refused: the missing device is what stops them."""
    outs, ins, call, same = overlap_cases(lib)[entry]
    every = {**ins, **outs}
    far = {name: (k + 1) << 36 for k, name in enumerate(every)}
    after = lambda i: far[i] + (every[i] + 15) // 16 * 16  # noqa: E731
    none = call(far)
    assert none not in (OK, INVALID, SHAPE, ALIGN, WORKSPACE)
    for o in outs:
        for i in every:
            if i != o:
                assert call({**far, o: after(i)}) == none, (o, i)
                assert call({**far, o: far[i] - (every[o] + 15) // 16 * 16}) == none, (o, i)
    for o, i in same:
        assert call({**far, o: far[i]}) == none, (o, i)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory: only where no kernel can be launched")
def test_abi_backward_over_what_is_not_read(lib):
    """A gradient may lie over an operand that only the other gradient reads, and over dh and gate_up."""
    A = [(k + 1) << 36 for k in range(6)]

    def call(dh=A[0], x=A[1], W=A[2], gu=A[3], dx=A[4], dW=A[5]):
        return lib.bsfp4_gated_ffn_backward(dh, x, W, gu, 0, dx, dW, M_, N_, K_, FAKE, 1 << 30, None)

    none = call()
    assert none not in (OK, INVALID)
    assert call(dx=A[1], dW=None) == call(dW=A[2], dx=None) == call(dx=A[0]) == call(dW=A[3]) == none
    assert call(dx=A[1]) == call(dW=A[2]) == call(dx=A[2], dW=None) == call(dW=A[1], dx=None) == INVALID
