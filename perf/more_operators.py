"""Measured cases of the 8-bit linear operators: RMS norm, gated activation and quantization with a scale for each token,
and the matrix product that reads them with a scale for each channel.  Each has a plain form in elementary torch
operations and the calls a user's program makes of this package (`own`)."""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
TOP = {"int8": 127.0, "e4m3": 448.0}
FLOOR = 2.0 ** -126  # the smallest step


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one user, one new token: residual and norm in front of a projection; latency
        {"name": "add norm one token h2560", "op": "norm", "dt": "bf16", "t": 1, "h": 2560, "add": True, "offset": 0},
        # a decode batch of a model with zero-centred norm weights
        {"name": "norm batch h2048", "op": "norm", "dt": "fp16", "t": 67, "h": 2048, "add": False, "offset": 1},
        # a chunk of prompt tokens
        {"name": "add norm chunk h4096", "op": "norm", "dt": "bf16", "t": 4096, "h": 4096, "add": True, "offset": 0},
        # the gate of a decode batch
        {"name": "silu gate batch d9728", "op": "glu", "dt": "bf16", "t": 64, "d": 9728, "act": "silu"},
        # the gate of a chunk of prompt tokens
        {"name": "gelu gate chunk d10240", "op": "glu", "dt": "bf16", "t": 4001, "d": 10240, "act": "gelu_tanh"},
        # attention outputs of 32 heads of 128 in front of the output projection: a small batch, and a chunk in fp32
        {"name": "quantize batch 32x128", "op": "quant", "dt": "fp16", "t": 33, "h": 4096},
        {"name": "quantize chunk 16x256", "op": "quant", "dt": "fp32", "t": 2500, "h": 4096},
        # QKV projection of one token, 32/8 heads of 128, with a bias
        {"name": "product qkv one token e4m3", "op": "product", "q": "e4m3", "dt": "bf16", "t": 1, "k": 2560, "n": 6144,
         "bias": True},
        # down projection of a decode batch
        {"name": "product down batch int8", "op": "product", "q": "int8", "dt": "bf16", "t": 64, "k": 9728, "n": 2560,
         "bias": False},
        # QKV projection of a prompt of odd length, 16/2 heads of 256
        {"name": "product qkv prompt e4m3", "op": "product", "q": "e4m3", "dt": "fp16", "t": 1201, "k": 2048, "n": 5120,
         "bias": False},
        # gate and up projection of a long chunk
        {"name": "product gate-up chunk int8", "op": "product", "q": "int8", "dt": "bf16", "t": 4096, "k": 2560,
         "n": 19456, "bias": False},
        # a whole feed-forward block: norm, gate and up product, gate, down product
        {"name": "feed-forward int8", "op": "ffn", "q": "int8", "dt": "bf16", "t": 1024, "h": 2560, "d": 9728},
    ]


def draw(rng):
    def span(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):
        """Most widths are multiples of 64, as models have them; others of 16 or 8, and odd ones."""
        w, of = span(lo, hi), rng.choice([64, 64, 64, 16, 8, 1])
        return max(of, w // of * of)

    op = rng.choice(["norm", "norm", "glu", "quant", "product", "product", "product", "product", "ffn"])
    dt = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "norm":
        return {"op": op, "dt": dt, "t": span(1, 4096), "h": width(48, 8192), "add": rng.random() < 0.6,
                "offset": rng.choice([0, 1])}
    if op == "glu":
        return {"op": op, "dt": dt, "t": span(1, 4096), "d": width(48, 10240),
                "act": rng.choice(["silu", "gelu_tanh"])}
    if op == "quant":
        return {"op": op, "dt": dt, "t": span(1, 4096), "h": width(48, 8192)}
    q = rng.choice(["int8", "e4m3"])
    if op == "product":
        k, n = width(48, 9728), width(24, 19456)
        most = min(4096, 150_000_000_000 // (k * n))
        if k % 16:  # rows that do not start on 16 bytes
            most = min(most, 512)
        return {"op": op, "q": q, "dt": dt, "t": span(1, max(2, most)), "k": k, "n": n, "bias": rng.random() < 0.3}
    return {"op": op, "q": q, "dt": dt, "t": span(1, 1024), "h": 64 * span(4, 40), "d": 64 * span(8, 152)}


# ---------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _activations(g, t, h):
    """Values of about unit size in which every 61st channel is much larger, as in front of a projection."""
    x = _normal(g, t, h)
    x[:, ::61] *= 12.0
    return x


def _codes(x, q):
    """x in 8 bits with a scale for each row, as a checkpoint holds weights."""
    top = x.abs().amax(-1, keepdim=True).clamp(min=1e-20) / TOP[q]
    y = x / top
    return (y.round().to(torch.int8) if q == "int8" else y.to(torch.float8_e4m3fn)), top[:, 0].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, t, dt = case["op"], case["t"], TYPES[case["dt"]]
    s = {"op": op, "case": case, "eps": 1e-6}
    if op == "norm":
        s["x"], s["residual"] = _activations(g, t, case["h"]).to(dt), (4.0 * _activations(g, t, case["h"])).to(dt)
        s["w"] = (0.1 * _normal(g, case["h"]) + (1.0 - case["offset"])).to(dt)
        shape = (t, case["h"])
    elif op == "glu":
        s["x"] = _activations(g, t, 2 * case["d"]).to(dt)
        shape = (t, case["d"])
    elif op == "quant":
        s["x"] = _activations(g, t, case["h"]).to(dt)
        shape = (t, case["h"])
    elif op == "product":
        s["a"], s["sa"] = _codes(_activations(g, t, case["k"]), case["q"])
        s["w"], s["sw"] = _codes(0.02 * _normal(g, case["n"], case["k"]), case["q"])
        s["bias"] = _normal(g, case["n"]).to(dt) if case["bias"] else None
        s["out"] = torch.empty((t, case["n"]), dtype=dt, device="cuda")
        return s
    else:
        h, d = case["h"], case["d"]
        s["x"], s["residual"] = _activations(g, t, h).to(dt), (4.0 * _activations(g, t, h)).to(dt)
        s["w"] = (0.1 * _normal(g, h) + 1.0).to(dt)
        s["up"], s["su"] = _codes(0.05 * _normal(g, 2 * d, h), case["q"])
        s["down"], s["sd"] = _codes(0.02 * _normal(g, h, d), case["q"])
        return s
    s["codes"] = torch.empty(shape, dtype=torch.uint8, device="cuda")
    s["scales"] = torch.empty(t, dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return _RUN[state["op"]](state)


def _eight(p, q):
    """Codes of the rows of p (fp32), and the step of each row."""
    most = p.abs().amax(-1, keepdim=True)
    top = torch.full_like(most, TOP[q])
    inv, step = (top / most).clamp(max=1.0 / FLOOR), (most / top).clamp(min=FLOOR)
    y = p * inv
    codes = y.round().to(torch.int8) if q == "int8" else y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes, step[:, 0]


def _add(x, residual):
    residual.copy_((x.float() + residual.float()).to(x.dtype))
    return residual


def _normed(x, w, offset, eps, q):
    f = x.float()
    r = torch.rsqrt(f.square().mean(-1) + eps)
    codes, step = _eight(f * (w.float() + offset), q)
    return codes, r * step


def _gated(x, act):
    gate, up = x.float().chunk(2, -1)
    if act == "silu":
        return gate / (1.0 + torch.exp(-gate)) * up
    z = math.sqrt(2.0 / math.pi) * (gate + 0.044715 * gate * gate * gate)
    return gate / (1.0 + torch.exp(-2.0 * z)) * up


def _product(a, w, sa, sw, bias, dt):
    y = (a.float() @ w.float().t()) * sa[:, None] * sw
    return (y if bias is None else y + bias.float()).to(dt)


def _norm(s):
    c = s["case"]
    if own:
        from memory_bound_decode_qk_gb300 import edge_ops

        if c["add"]:
            edge_ops.add_rmsnorm_q8(s["x"], s["residual"], s["w"], eps=s["eps"], weight_offset=c["offset"], fp8=True,
                                    out=s["codes"], scales=s["scales"])
            return s["codes"].view(torch.float8_e4m3fn), s["scales"], s["residual"]
        edge_ops.rmsnorm_q8(s["x"], s["w"], eps=s["eps"], weight_offset=c["offset"], fp8=True, out=s["codes"],
                            scales=s["scales"])
        return s["codes"].view(torch.float8_e4m3fn), s["scales"]
    x = _add(s["x"], s["residual"]) if c["add"] else s["x"]
    codes, scales = _normed(x, s["w"], c["offset"], s["eps"], "e4m3")
    return (codes, scales, x) if c["add"] else (codes, scales)


def _glu(s):
    if own:
        from memory_bound_decode_qk_gb300 import edge_ops

        edge_ops.glu_act_q8(s["x"], s["case"]["act"], fp8=True, out=s["codes"], scales=s["scales"])
        return s["codes"].view(torch.float8_e4m3fn), s["scales"]
    return _eight(_gated(s["x"], s["case"]["act"]), "e4m3")


def _quant(s):
    if own:
        from memory_bound_decode_qk_gb300 import edge_ops

        edge_ops.quantize_q8(s["x"], fp8=True, out=s["codes"], scales=s["scales"])
        return s["codes"].view(torch.float8_e4m3fn), s["scales"]
    return _eight(s["x"].float(), "e4m3")


def _one_product(s):
    if own:
        from memory_bound_decode_qk_gb300 import edge_ops

        return edge_ops.matmul_q8(s["a"], s["w"], s["sa"], s["sw"], bias=s["bias"], dtype=s["out"].dtype, out=s["out"])
    return _product(s["a"], s["w"], s["sa"], s["sw"], s["bias"], s["out"].dtype)


def _ffn(s):
    q, dt = s["case"]["q"], s["x"].dtype
    if own:
        from memory_bound_decode_qk_gb300 import edge_ops

        fp8 = q == "e4m3"
        a, sa = edge_ops.add_rmsnorm_q8(s["x"], s["residual"], s["w"], eps=s["eps"], fp8=fp8)
        y = edge_ops.matmul_q8(a, s["up"], sa, s["su"], dtype=dt)
        a, sa = edge_ops.glu_act_q8(y, "silu", fp8=fp8)
        return edge_ops.matmul_q8(a, s["down"], sa, s["sd"], dtype=dt), s["residual"]
    x = _add(s["x"], s["residual"])
    a, sa = _normed(x, s["w"], 0, s["eps"], q)
    y = _product(a, s["up"], sa, s["su"], None, dt)
    a, sa = _eight(_gated(y, "silu"), q)
    return _product(a, s["down"], sa, s["sd"], None, dt), x


_RUN = {"norm": _norm, "glu": _glu, "quant": _quant, "product": _one_product, "ffn": _ffn}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, t, size = case["op"], case["t"], SIZE[case["dt"]]
    if op == "norm":
        h = case["h"]
        return {"bytes": t * h * (size * (3 if case["add"] else 1) + 1) + 4 * t + h * size, "flops": 6 * t * h}
    if op == "glu":
        return {"bytes": t * case["d"] * (2 * size + 1) + 4 * t, "flops": 10 * t * case["d"]}
    if op == "quant":
        return {"bytes": t * case["h"] * (size + 1) + 4 * t, "flops": 3 * t * case["h"]}
    if op == "product":
        k, n = case["k"], case["n"]
        return {"bytes": (t + n) * (k + 4) + t * n * size + (n * size if case["bias"] else 0), "flops": 2 * t * n * k}
    h, d = case["h"], case["d"]
    return {"bytes": 4 * t * h * size + h * size + 3 * h * d + 4 * (2 * d + h), "flops": 6 * t * h * d}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "glu": _exact_glu, "quant": _exact_quant, "product": _exact_product,
            "ffn": _exact_ffn}[case["op"]](case, s)


def _steps(v, q):
    """The step of each row of v (64 bits), and the row in these steps before it is rounded to codes."""
    step = torch.maximum(v.abs().max(dim=1).values / TOP[q], torch.tensor(FLOOR, dtype=torch.float64, device=v.device))
    return v / step.unsqueeze(1), step


def _norm_steps(x, w, offset, eps, q):
    v, step = _steps(x.double() * (w.double() + offset), q)
    return v, step / (x.double().pow(2).sum(1) / x.shape[1] + eps).sqrt()


def _gate64(x, act):
    n = x.shape[1] // 2
    a, b = x[:, :n].double(), x[:, n:].double()
    if act == "silu":
        return a * torch.special.expit(a) * b
    return 0.5 * a * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (a + 0.044715 * a ** 3))) * b


def _exact_norm(case, s):
    if not case["add"]:
        return _norm_steps(s["x"], s["w"], case["offset"], s["eps"], "e4m3")
    total = (s["x"].double() + s["residual"].double()).to(s["x"].dtype)
    return *_norm_steps(total, s["w"], case["offset"], s["eps"], "e4m3"), total.double()


def _exact_glu(case, s):
    return _steps(_gate64(s["x"], case["act"]), "e4m3")


def _exact_quant(case, s):
    return _steps(s["x"].double(), "e4m3")


def _times(a, w, sa, sw):
    return torch.einsum("tk,nk->tn", a.double(), w.double()) * torch.outer(sa.double(), sw.double())


def _exact_product(case, s):
    y = _times(s["a"], s["w"], s["sa"], s["sw"])
    return y if s["bias"] is None else y + s["bias"].double().unsqueeze(0)


def _nearest(v, q):
    return torch.round(v) if q == "int8" else v.to(torch.float8_e4m3fn).double()


def _exact_ffn(case, s):
    q, dt = case["q"], s["x"].dtype
    total = (s["x"].double() + s["residual"].double()).to(dt)
    v, sa = _norm_steps(total, s["w"], 0, s["eps"], q)
    y = _times(_nearest(v, q), s["up"], sa, s["su"]).to(dt)
    v, sa = _steps(_gate64(y, "silu"), q)
    return _times(_nearest(v, q), s["down"], sa, s["sd"]), total.double()
