"""What is measured of the feed-forward block's operators: 8-bit integer products, the gated
feed-forward product and the norms around a block.

Kinds of case:
  int8_linear   bf16 activations quantised per token to 8-bit integers, times 8-bit weights with
                one scale per output channel, plus a bias
  int8_gated    the same activations and weights through the gated product: act(gate) * up
  gated         the gated product in bf16 (serving)
  gated_train   the gated product in bf16 with its backward pass (training)
  norm          post-norm, gate, residual add and the next block's pre-norm in one pass (serving);
                "int8" gives the pre-norm's rows quantised per token
  norm_train    the same in bf16 with its backward pass
Rows are tokens.  Weight matrices are [outputs, inputs]; a gated weight holds the gate rows, then
the up rows.
"""
import math

import torch

own = False

EPS = 1e-6


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of one sequence through an 8-bit projection: launch and weight-read latency
        {"name": "int8_linear_decode", "kind": "int8_linear", "M": 1, "N": 4096, "K": 7168, "bias": True},
        # a small ragged batch of prompts through a wide 8-bit projection
        {"name": "int8_linear_ragged", "kind": "int8_linear", "M": 250, "N": 14336, "K": 4096, "bias": False},
        # a long prompt: the compute-bound product
        {"name": "int8_linear_prefill", "kind": "int8_linear", "M": 4096, "N": 4096, "K": 7168, "bias": True},
        # a handful of concurrent sequences decoding through 8-bit gate and up projections
        {"name": "int8_gated_decode", "kind": "int8_gated", "M": 5, "H": 4096, "I": 7168, "act": "silu"},
        # a prompt chunk of odd length through the same layer
        {"name": "int8_gated_prefill", "kind": "int8_gated", "M": 1003, "H": 4096, "I": 7168, "act": "silu"},
        # one token through a bf16 gated layer
        {"name": "gated_decode", "kind": "gated", "M": 1, "H": 4096, "I": 7168, "act": "silu"},
        # a middling batch, odd token count and an odd width, another activation
        {"name": "gated_batch", "kind": "gated", "M": 333, "H": 2048, "I": 1544, "act": "gelu_tanh"},
        # a small layer's training step, ragged sizes
        {"name": "gated_train_ragged", "kind": "gated_train", "M": 777, "H": 2048, "I": 776, "act": "gelu"},
        # a large layer's training step: the largest case
        {"name": "gated_train_large", "kind": "gated_train", "M": 4096, "H": 4096, "I": 7168, "act": "silu"},
        # one token between two blocks, the next block taking 8-bit activations
        {"name": "norm_decode_int8", "kind": "norm", "T": 1, "H": 4096, "groups": 1, "fmt": "int8"},
        # a prompt between two blocks, a gate per sequence
        {"name": "norm_prefill", "kind": "norm", "T": 4000, "H": 7168, "groups": 8, "fmt": "bf16"},
        # a training step's norms with a gate per channel
        {"name": "norm_train", "kind": "norm_train", "T": 8192, "H": 4096, "groups": 1},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    """One more case of the listed ranges; costs are held under the largest listed of its kind."""
    kind = rng.choice(["int8_linear", "int8_gated", "gated", "gated_train", "norm", "norm_train"])
    act = rng.choice(["silu", "gelu", "gelu_tanh"])
    if kind == "int8_linear":
        return {"kind": kind, "M": _log(rng, 1, 4096), "N": _log(rng, 512, 4096, 8),
                "K": _log(rng, 512, 7168, 16), "bias": rng.random() < 0.5}
    if kind == "int8_gated":
        return {"kind": kind, "M": _log(rng, 1, 1003), "H": _log(rng, 512, 4096, 16),
                "I": _log(rng, 256, 7168, 8), "act": act}
    if kind == "gated":
        return {"kind": kind, "M": _log(rng, 1, 2048), "H": _log(rng, 512, 4096, 8),
                "I": _log(rng, 256, 7168, 8), "act": act}
    if kind == "gated_train":
        return {"kind": kind, "M": _log(rng, 64, 4096), "H": _log(rng, 512, 4096, 8),
                "I": _log(rng, 256, 7168, 8), "act": act}
    groups = rng.choice([1, 1, 2, 3, 8])
    if kind == "norm":
        return {"kind": kind, "T": groups * _log(rng, 1, 4000 // groups), "H": _log(rng, 512, 7168, 8),
                "groups": groups, "fmt": rng.choice(["bf16", "int8"])}
    return {"kind": kind, "T": groups * _log(rng, 16, 8192 // groups), "H": _log(rng, 512, 4096, 8), "groups": groups}


# ----------------------------------------------------------------------------- inputs

class _Inputs:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=self.g, device="cuda") * std + mean).to(dtype)

    def activations(self, M, K):
        """Hidden states: N(0, 1) with a few channels of much larger values, as trained models have them."""
        x = torch.randn((M, K), generator=self.g, device="cuda")
        hot = torch.randint(0, K, (max(1, K // 512),), generator=self.g, device="cuda")
        x[:, hot] *= 12.0
        return x.to(torch.bfloat16)

    def int8_weight(self, N, K):
        """N(0, 0.02) weights as 8-bit integers with one scale per row."""
        w = torch.randn((N, K), generator=self.g, device="cuda") * 0.02
        s = w.abs().amax(dim=1) / 127.0
        return torch.round(w / s[:, None]).to(torch.int8), s


def prepare(case, seed):
    inp = _Inputs(seed)
    st = {"case": dict(case)}
    kind = case["kind"]
    if kind == "int8_linear":
        st["x"] = inp.activations(case["M"], case["K"])
        st["w"], st["ws"] = inp.int8_weight(case["N"], case["K"])
        st["bias"] = inp.normal((case["N"],), 0.5) if case["bias"] else None
    elif kind == "int8_gated":
        st["x"] = inp.activations(case["M"], case["H"])
        st["w"], st["ws"] = inp.int8_weight(2 * case["I"], case["H"])
    elif kind in ("gated", "gated_train"):
        st["x"] = inp.activations(case["M"], case["H"])
        st["w"] = inp.normal((2 * case["I"], case["H"]), 0.02)
        if kind == "gated_train":
            st["dh"] = inp.normal((case["M"], case["I"]), 1e-2)
    else:
        T, H = case["T"], case["H"]
        st["x"] = inp.activations(T, H)
        st["residual"] = inp.normal((T, H), 3.0)
        st["w_post"] = inp.normal((H,), 0.2, 1.0)
        st["w_pre"] = inp.normal((H,), 0.2, 1.0)
        st["gate"] = inp.normal((case["groups"], H), 0.5, 0.3)
        st["scale"] = 0.5
        if kind == "norm_train":
            st["dres"] = inp.normal((T, H), 1e-2)
            st["dz"] = inp.normal((T, H), 1e-2)
    return st


# ----------------------------------------------------------------------------- plain forms

def _act(name, g):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    if name == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(name, g):
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)


def _int8_rows(x):
    """Each row's 8-bit integers, round-to-even of 127 x / max|x|, and its scale max|x| / 127.  In 64
    bits: the quotient of bf16 values is often exactly half-way between two integers."""
    xd = x.double()
    amax = xd.abs().amax(dim=1, keepdim=True)
    q = torch.round(127.0 * xd / torch.where(amax == 0, 1.0, amax))
    return q.to(torch.int8), (amax[:, 0] / 127.0).float()


def _int8_product(st):
    q, s = _int8_rows(st["x"])
    return (q.float() @ st["w"].float().t()) * s[:, None] * st["ws"][None, :]


def _rstd(x):
    """1 / rms of each row; the mean square in 64 bits, as the rows' roundings hang on it."""
    xd = x.double()
    return (1.0 / torch.sqrt((xd * xd).mean(dim=1, keepdim=True) + EPS)).float()


def _norm(st):
    x, r, gate = st["x"], st["residual"], st["gate"]
    g = gate.float().repeat_interleave(r.shape[0] // gate.shape[0], dim=0) * st["scale"]
    n = x.float() * _rstd(x) * st["w_post"].float()
    res = (r.float() + g * n).to(torch.bfloat16)
    z = (res.float() * _rstd(res) * st["w_pre"].float()).to(torch.bfloat16)
    return res, z


def _norm_back(st, res):
    T, H = res.shape
    G = st["gate"].shape[0]
    scale = st["scale"]
    dz, w_pre, w_post = st["dz"].float(), st["w_pre"].float(), st["w_post"].float()
    g = st["gate"].float().repeat_interleave(T // G, dim=0) * scale
    rs = _rstd(res)
    zh = res.float() * rs
    gz = dz * w_pre
    d = st["dres"].float() + rs * (gz - zh * (gz * zh).mean(dim=1, keepdim=True))
    dw_pre = (dz * zh).sum(dim=0)
    xs = _rstd(st["x"])
    xh = st["x"].float() * xs
    dn = d * g
    dw_post = (dn * xh).sum(dim=0)
    dgate = (d * xh * w_post * scale).view(G, T // G, H).sum(dim=1)
    gx = dn * w_post
    dx = xs * (gx - xh * (gx * xh).mean(dim=1, keepdim=True))
    return {"dx": dx.to(torch.bfloat16), "dres": d.to(torch.bfloat16), "dw_post": dw_post, "dw_pre": dw_pre,
            "dgate": dgate}


def _plain(st):
    case = st["case"]
    kind = case["kind"]
    if kind == "int8_linear":
        d = _int8_product(st)
        if st["bias"] is not None:
            d = d + st["bias"].float()
        return d.to(torch.bfloat16)
    if kind == "int8_gated":
        gate, up = _int8_product(st).split(case["I"], dim=1)
        return (_act(case["act"], gate) * up).to(torch.bfloat16)
    if kind in ("gated", "gated_train"):
        x, w = st["x"].float(), st["w"].float()
        gate, up = (x @ w.t()).split(case["I"], dim=1)
        h = (_act(case["act"], gate) * up).to(torch.bfloat16)
        if kind == "gated":
            return h
        dh = st["dh"].float()
        dgu = torch.cat([dh * up * _act_grad(case["act"], gate), dh * _act(case["act"], gate)], dim=1)
        return {"h": h, "dx": (dgu @ w).to(torch.bfloat16), "dw": (dgu.t() @ x).to(torch.bfloat16)}
    if kind == "norm":
        res, z = _norm(st)
        if case["fmt"] == "bf16":
            return {"res": res, "z": z}
        q, s = _int8_rows(z)
        return {"res": res, "q": q, "s": s}
    res, z = _norm(st)
    return {"res": res, "z": z, **_norm_back(st, res)}


# ----------------------------------------------------------------------------- the framework's calls

def _own(st):
    import block_scaled_fp4_e2m1_amd as bs
    case = st["case"]
    kind = case["kind"]
    if kind == "int8_linear":
        return bs.int8_quantize_gemm(st["x"], st["w"], st["ws"], bias=st["bias"])
    if kind == "int8_gated":
        q, s = bs.int8_quantize(st["x"])
        return bs.int8_gated_ffn(q, s, st["w"], st["ws"], act=case["act"])
    if kind == "gated":
        return bs.gated_ffn(st["x"], st["w"], act=case["act"])
    if kind == "gated_train":
        h, gate_up = bs.gated_ffn(st["x"], st["w"], act=case["act"], save_gate_up=True)
        dx, dw = bs.gated_ffn_backward(st["dh"], st["x"], st["w"], gate_up, act=case["act"])
        return {"h": h, "dx": dx, "dw": dw}
    norm = dict(w_post=st["w_post"], w_pre=st["w_pre"], gate=st["gate"], scale=st["scale"], eps=EPS)
    if kind == "norm":
        if case["fmt"] == "bf16":
            res, z = bs.block_norm(st["x"], st["residual"], **norm)
            return {"res": res, "z": z}
        res, q, s = bs.block_norm(st["x"], st["residual"], fmt="int8", **norm)
        return {"res": res, "q": q, "s": s}
    res, z = bs.block_norm(st["x"], st["residual"], **norm)
    dx, dres, dw_post, dw_pre, dgate = bs.block_norm_backward(st["dres"], st["dz"], st["x"], res, **norm)
    return {"res": res, "z": z, "dx": dx, "dres": dres, "dw_post": dw_post, "dw_pre": dw_pre, "dgate": dgate}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ----------------------------------------------------------------------------- least work

def work(case):
    kind = case["kind"]
    if kind == "int8_linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K + 4 * N + 2 * M * N + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    if kind in ("int8_gated", "gated", "gated_train"):
        M, H, I = case["M"], case["H"], case["I"]
        one = 2 * M * (2 * I) * H
        if kind == "int8_gated":
            return {"bytes": 2 * M * H + 2 * I * H + 8 * I + 2 * M * I, "flops": one}
        if kind == "gated":
            return {"bytes": 2 * M * H + 4 * I * H + 2 * M * I, "flops": one}
        # x, W, dh in; h, dx, dW out; three products
        return {"bytes": 2 * (2 * M * H + 2 * M * I) + 2 * (4 * I * H), "flops": 3 * one}
    T, H, G = case["T"], case["H"], case["groups"]
    small = 4 * H + 2 * G * H
    if kind == "norm":
        z = 2 * T * H if case["fmt"] == "bf16" else T * H + 4 * T
        return {"bytes": 6 * T * H + z + small, "flops": 12 * T * H}
    # x, residual, dres, dz in; res, z, dx, dresidual out, and the three weight gradients
    return {"bytes": 16 * T * H + small + 4 * (2 * H + G * H), "flops": 40 * T * H}


# ----------------------------------------------------------------------------- 64 bits

def _bf16(v):
    return v.to(torch.bfloat16).double()


def _exact_act(name, v):
    """act(v) and act'(v) in 64 bits."""
    if name == "silu":
        s = torch.sigmoid(v)
        return v * s, s + v * s * (1 - s)
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-v / math.sqrt(2.0))
        return v * cdf, cdf + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    # 0.5 (1 + tanh u) = sigmoid(2 u)
    k = math.sqrt(8.0 / math.pi)
    s = torch.sigmoid(k * (v + 0.044715 * v ** 3))
    return v * s, s + v * s * (1 - s) * k * (1 + 0.134145 * v ** 2)


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    x = st["x"].double()
    if kind in ("int8_linear", "int8_gated"):
        top = x.abs().max(dim=1, keepdim=True).values
        codes = (x * 127 / top.clamp_min(1e-300)).round()
        y = torch.mm(codes, st["w"].double().t()) * (top / 127) * st["ws"].double()
        if kind == "int8_linear":
            return y if st["bias"] is None else y + st["bias"].double()
        return _exact_act(case["act"], y[:, :case["I"]])[0] * y[:, case["I"]:]
    if kind in ("gated", "gated_train"):
        wg, wu = st["w"].double().chunk(2)
        g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
        a, da = _exact_act(case["act"], g)
        if kind == "gated":
            return a * u
        dh = st["dh"].double()
        dg, du = dh * u * da, dh * a
        return {"h": a * u, "dx": torch.mm(dg, wg) + torch.mm(du, wu),
                "dw": torch.cat([torch.mm(dg.t(), x), torch.mm(du.t(), x)])}
    T, H, G = case["T"], case["H"], case["groups"]
    wp, wn = st["w_post"].double(), st["w_pre"].double()
    gate = (st["gate"].double() * st["scale"])[:, None, :].expand(G, T // G, H).reshape(T, H)
    inv_x = (x.square().mean(1, keepdim=True) + EPS).rsqrt()
    # the residual stream is kept in bf16, and the next norm reads what is kept
    kept_wide = st["residual"].double() + gate * (x * inv_x * wp)
    kept = _bf16(kept_wide)
    inv_r = (kept.square().mean(1, keepdim=True) + EPS).rsqrt()
    z = kept * inv_r * wn
    if kind == "norm":
        if case["fmt"] == "bf16":
            return {"res": kept_wide, "z": z}
        return {"res": kept_wide, "q": None, "s": _bf16(z).abs().amax(1) / 127}
    dz = st["dz"].double()
    t = dz * wn
    d = st["dres"].double() + inv_r * t - kept * inv_r ** 3 * (t * kept).sum(1, keepdim=True) / H
    e = d * gate * wp
    dx = inv_x * e - x * inv_x ** 3 * (e * x).sum(1, keepdim=True) / H
    return {"res": kept_wide, "z": z, "dx": dx, "dres": d, "dw_post": (d * gate * x * inv_x).sum(0),
            "dw_pre": (dz * kept * inv_r).sum(0),
            "dgate": (d * x * inv_x * wp * st["scale"]).reshape(G, T // G, H).sum(1)}
