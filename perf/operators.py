"""The feed-forward operators as measured work: the cases, their inputs, one pass of each, and what a pass costs.

Four operators of a transformer's feed-forward block:

  quantize  int8 codes of activations with one scale for each token,
  gemm      the product of int8 activations and int8 weights with a scale for each token and each channel,
  gated     the gated product act(x Wg^T) * (x Wu^T) of such int8 operands,
  ffn       the same gated product of bf16 operands, alone (serving) or with its backward pass (training).

``run`` computes them with elementary torch operations, or, where ``own`` is true, with this repository's
kernels.
"""
import math

import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One token of a decode step entering a 4096-wide block: all latency.
        {"name": "quantize 1x4096 bf16", "op": "quantize", "rows": 1, "k": 4096, "type": "bf16"},
        # The hidden activations of 333 prompt tokens before the down projection.
        {"name": "quantize 333x14336 bf16", "op": "quantize", "rows": 333, "k": 14336, "type": "bf16"},
        # A whole batch of fp32 activations, the size of the repository's quantizer workload.
        {"name": "quantize 8192x8192 f32", "op": "quantize", "rows": 8192, "k": 8192, "type": "f32"},
        # Eight sequences decoding through an up projection (the decode GEMV workload's size).
        {"name": "gemm 8x14336x4096", "op": "gemm", "m": 8, "n": 14336, "k": 4096, "out": "bf16"},
        # A short prompt through a square projection (the W4A8 workload's size).
        {"name": "gemm 256x8192x8192", "op": "gemm", "m": 256, "n": 8192, "k": 8192, "out": "bf16"},
        # A projection with no even size, fp32 results.
        {"name": "gemm 1003x1117x1040 f32", "op": "gemm", "m": 1003, "n": 1117, "k": 1040, "out": "f32"},
        # A long prefill through a square projection (the MXFP4 GEMM workload's size).
        {"name": "gemm 8192x8192x8192", "op": "gemm", "m": 8192, "n": 8192, "k": 8192, "out": "bf16"},
        # One token of one sequence through the gated half of a feed-forward block.
        {"name": "gated 1x14336x4096 silu", "op": "gated", "m": 1, "n": 14336, "k": 4096, "act": "silu", "out": "bf16"},
        # A prefill chunk through the same block.
        {"name": "gated 2048x14336x4096 gelu_tanh", "op": "gated", "m": 2048, "n": 14336, "k": 4096, "act": "gelu_tanh",
         "out": "bf16"},
        # Sixteen sequences decoding through the unquantized block.
        {"name": "ffn 16x14336x4096 silu", "op": "ffn", "m": 16, "n": 14336, "k": 4096, "act": "silu", "train": False},
        # A small training step with ragged sizes.
        {"name": "ffn train 301x1003x520 gelu", "op": "ffn", "m": 301, "n": 1003, "k": 520, "act": "gelu", "train": True},
        # A training step of 8192 tokens.
        {"name": "ffn train 8192x14336x4096 silu", "op": "ffn", "m": 8192, "n": 14336, "k": 4096, "act": "silu",
         "train": True},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in lo..hi, even over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gated", "ffn"])
    if op == "quantize":
        return {"op": op, "rows": _spread(rng, 1, 8192), "k": _spread(rng, 128, 16384, 16),
                "type": rng.choice(["bf16", "f32"])}
    m, n = _spread(rng, 1, 8192), _spread(rng, 128, 14336)
    if op == "gemm":
        return {"op": op, "m": m, "n": n, "k": _spread(rng, 128, 14336, 16), "out": rng.choice(["bf16", "f32"])}
    act = rng.choice(["silu", "gelu", "gelu_tanh"])
    if op == "gated":
        return {"op": op, "m": m, "n": n, "k": _spread(rng, 128, 8192, 16), "act": act,
                "out": rng.choice(["bf16", "f32"])}
    return {"op": op, "m": m, "n": n, "k": _spread(rng, 128, 4096, 8), "act": act, "train": rng.random() < 0.6}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def codes(rows, k):
        # Rows of a normal distribution quantized by their own maximum have about this spread.
        return (normal(rows, k) * 34).round().clamp(-127, 127).to(torch.int8)

    def scales(rows, typical):
        return (normal(rows) * 0.3).exp() * typical

    state = {"case": case}
    if case["op"] == "quantize":
        # Activations: tokens of different magnitude, and a few channels far above the others.
        x = normal(case["rows"], case["k"]) * (normal(case["rows"], 1) * 0.5).exp()
        x *= 1 + 20 * (torch.rand(case["k"], generator=g, device=DEV) < 0.004)
        state["x"] = x.to(TYPES[case["type"]])
        return state
    m, n, k = case["m"], case["n"], case["k"]
    if case["op"] == "gemm":
        state |= {"a": codes(m, k), "sa": scales(m, 0.03), "b": codes(n, k), "sb": scales(n, 0.0005)}
    elif case["op"] == "gated":
        # The scales give pre-activations of about unit size: sqrt(k) * 34^2 * sa * sg.
        s = 1 / (34 * 34 * math.sqrt(k) * 0.03)
        state |= {"a": codes(m, k), "sa": scales(m, 0.03), "bg": codes(n, k), "sg": scales(n, s),
                  "bu": codes(n, k), "su": scales(n, s)}
    else:
        state |= {"x": normal(m, k).bfloat16(), "wg": (normal(n, k) / math.sqrt(k)).bfloat16(),
                  "wu": (normal(n, k) / math.sqrt(k)).bfloat16()}
        if case["train"]:
            state["dh"] = (normal(m, n) * 0.01).bfloat16()
    return state


def _gate(g, act):
    """The activation of g and its derivative, in g's type."""
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    if act == "silu":
        z, dz = g, 1.0
    else:
        c = 2 * math.sqrt(2 / math.pi)
        z, dz = c * (g + 0.044715 * g * g * g), c * (1 + 3 * 0.044715 * g * g)
    s = 1 / (1 + torch.exp(-z))
    return g * s, s + g * s * (1 - s) * dz


def _plain(s, case):
    op = case["op"]
    if op == "quantize":
        x = s["x"].float()
        most = x.abs().amax(dim=1)
        scale = most / torch.full_like(most, 127)
        inverse = (torch.ones_like(scale) / scale).clamp(max=torch.finfo(torch.float32).max)
        return (x * inverse[:, None]).round().clamp(-127, 127).to(torch.int8), scale
    if op == "gemm":
        d = s["a"].float() @ s["b"].float().t()
        return (d * s["sa"][:, None] * s["sb"][None, :]).to(TYPES[case["out"]])
    if op == "gated":
        a = s["a"].float()
        g = a @ s["bg"].float().t() * s["sa"][:, None] * s["sg"][None, :]
        u = a @ s["bu"].float().t() * s["sa"][:, None] * s["su"][None, :]
        return (_gate(g, case["act"])[0] * u).to(TYPES[case["out"]])
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a, da = _gate(g, case["act"])
    h = (a * u).bfloat16()
    if not case["train"]:
        return h
    dh = s["dh"].float()
    dg, du = dh * u * da, dh * a
    return {"h": h, "dx": (dg @ wg + du @ wu).bfloat16(), "dwg": (dg.t() @ x).bfloat16(), "dwu": (du.t() @ x).bfloat16()}


def _own(s, case):
    import block_scaled_precision_e2m1_amd as fp4

    op = case["op"]
    if op == "quantize":
        return fp4.int8_quantize(s["x"])
    if op == "gemm":
        return fp4.w8a8_gemm(s["a"], s["sa"], s["b"], s["sb"], out_dtype=TYPES[case["out"]])
    if op == "gated":
        return fp4.w8a8_gated_gemm(s["a"], s["sa"], s["bg"], s["sg"], s["bu"], s["su"], act=case["act"],
                                   out_dtype=TYPES[case["out"]])
    if not case["train"]:
        return fp4.gated_gemm(s["x"], s["wg"], s["wu"], act=case["act"])
    h, g, u = fp4.gated_gemm(s["x"], s["wg"], s["wu"], act=case["act"], save=True)
    dx, dwg, dwu = fp4.gated_gemm_backward(s["dh"], s["x"], s["wg"], s["wu"], g, u, act=case["act"])
    return {"h": h, "dx": dx, "dwg": dwg, "dwu": dwu}


def run(state):
    return _own(state, state["case"]) if own else _plain(state, state["case"])


def work(case):
    op = case["op"]
    if op == "quantize":
        rows, k = case["rows"], case["k"]
        return {"bytes": rows * k * (2 if case["type"] == "bf16" else 4) + rows * k + 4 * rows, "flops": 3 * rows * k}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "gemm":
        return {"bytes": m * k + n * k + 4 * (m + n) + m * n * (2 if case["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    if op == "gated":
        return {"bytes": m * k + 2 * n * k + 4 * (m + 2 * n) + m * n * (2 if case["out"] == "bf16" else 4),
                "flops": 4 * m * n * k}
    if not case["train"]:
        return {"bytes": 2 * (m * k + 2 * n * k + m * n), "flops": 4 * m * n * k}
    # x, wg, wu, dh read; h, dx, dwg, dwu written; two products forward and four backward.
    return {"bytes": 2 * (m * k + 2 * n * k + m * n) + 2 * (m * n + m * k + 2 * n * k), "flops": 12 * m * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        # The definition rounds the scale, its inverse and each product to 32 bits: products and quotients of
        # 32-bit values are formed in 64 bits here and rounded to 32.
        x = s["x"].double()
        scale = (x.abs().max(dim=1).values / x.new_full((), 127)).float().double()
        inverse = scale.reciprocal().float().double()
        return torch.mul(x, inverse.unsqueeze(1)).float().double().round().clamp(-127, 127).to(torch.int8), scale
    f = torch.nn.functional
    act = {"silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda t: f.gelu(t, approximate="tanh")}
    if op == "gemm":
        return torch.mm(s["a"].double() * s["sa"].double().unsqueeze(1), (s["b"].double() * s["sb"].double().unsqueeze(1)).T)
    if op == "gated":
        a = s["a"].double() * s["sa"].double().unsqueeze(1)
        g = torch.mm(a, (s["bg"].double() * s["sg"].double().unsqueeze(1)).T)
        u = torch.mm(a, (s["bu"].double() * s["su"].double().unsqueeze(1)).T)
        return act[case["act"]](g) * u
    x, wg, wu = (s[name].double().requires_grad_(case["train"]) for name in ("x", "wg", "wu"))
    h = act[case["act"]](f.linear(x, wg)) * f.linear(x, wu)
    if not case["train"]:
        return h
    dx, dwg, dwu = torch.autograd.grad(h, (x, wg, wu), s["dh"].double())
    return {"h": h.detach(), "dx": dx, "dwg": dwg, "dwu": dwu}
