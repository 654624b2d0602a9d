"""What stands around a language model's products, as measured work: the cases, their inputs, one pass of each, and what a pass costs.

Three operators next to the products of this repository:

  norm      the root-mean-square norm of a row, with the residual's addition, its results in the rows' type or as int8
            or e4m3 codes with a scale for each row (what the int8 and W4A8 products take), alone or with its gradients,
  loss      the softmax cross entropy of X W^T against a token of the vocabulary for each row, without the logits in
            memory, alone or with its gradients,
  adapters  the low-rank products of many requests, each with an adapter of its own, added to what a projection that
            they share has given.

``run`` computes them with elementary torch operations, or, where ``own`` is true, with this repository's
kernels.
"""
import math

import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
IGNORE = -100
TOP = {"int8": 127, "e4m3": 448}


def listed():
    return [
        # One token of a decode step entering a 4096-wide block: all latency.
        {"name": "norm 1x4096 bf16", "op": "norm", "rows": 1, "k": 4096, "type": "bf16", "residual": True,
         "out": "same", "train": False},
        # Sixteen sequences decoding into an int8 projection.
        {"name": "norm 16x8192 int8", "op": "norm", "rows": 16, "k": 8192, "type": "bf16", "residual": True,
         "out": "int8", "train": False},
        # A prefill chunk into a W4A8 projection.
        {"name": "norm 4096x4096 e4m3", "op": "norm", "rows": 4096, "k": 4096, "type": "bf16", "residual": True,
         "out": "e4m3", "train": False},
        # The heads of 4096 tokens' queries, each normed by itself.
        {"name": "norm 131072x128 bf16", "op": "norm", "rows": 131072, "k": 128, "type": "bf16", "residual": False,
         "out": "same", "train": False},
        # A training step's norm with no even size, in fp32.
        {"name": "norm train 1003x1117 f32", "op": "norm", "rows": 1003, "k": 1117, "type": "f32", "residual": True,
         "out": "same", "train": True},
        # A training step of 8192 tokens.
        {"name": "norm train 8192x8192 bf16", "op": "norm", "rows": 8192, "k": 8192, "type": "bf16", "residual": True,
         "out": "same", "train": True},
        # A small training step with ragged sizes.
        {"name": "loss train 301x1003x520", "op": "loss", "m": 301, "v": 1003, "k": 520, "ignored": 0.1, "train": True},
        # Scoring one candidate token for each of sixteen sequences.
        {"name": "loss 16x131072x4096", "op": "loss", "m": 16, "v": 131072, "k": 4096, "ignored": 0.0, "train": False},
        # Fine-tuning on the answers alone: the half of the tokens that are prompts has no loss; an odd vocabulary.
        {"name": "loss train 4096x50021x2048", "op": "loss", "m": 4096, "v": 50021, "k": 2048, "ignored": 0.5,
         "train": True},
        # A training step of 8192 tokens over a large vocabulary.
        {"name": "loss train 8192x131072x4096", "op": "loss", "m": 8192, "v": 131072, "k": 4096, "ignored": 0.0,
         "train": True},
        # Thirty-two sequences decoding, each with one of 64 adapters.
        {"name": "adapters 32x4096x4096 r16", "op": "adapters", "m": 32, "n": 4096, "k": 4096, "r": 16, "l": 64,
         "requests": 32, "type": "bf16"},
        # Prompts of eight requests through an up projection.
        {"name": "adapters 4096x14336x4096 r64", "op": "adapters", "m": 4096, "n": 14336, "k": 4096, "r": 64, "l": 16,
         "requests": 8, "type": "bf16"},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in lo..hi, even over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "norm", "loss", "adapters"])
    if op == "norm":
        out = rng.choice(["same", "same", "int8", "e4m3"])
        k = _spread(rng, 64, 16384, 1 if out == "same" else 16)
        return {"op": op, "rows": _spread(rng, 1, min(131072, 8192 * 8192 // k)), "k": k,
                "type": rng.choice(["bf16", "f32"]), "residual": rng.random() < 0.7, "out": out,
                "train": out == "same" and rng.random() < 0.5}
    if op == "loss":
        return {"op": op, "m": _spread(rng, 1, 8192), "v": _spread(rng, 128, 131072), "k": _spread(rng, 64, 4096, 8),
                "ignored": rng.choice([0.0, 0.1, 0.5]), "train": rng.random() < 0.7}
    m = _spread(rng, 1, 4096)
    return {"op": op, "m": m, "n": _spread(rng, 64, 14336), "k": _spread(rng, 64, 8192, 8), "r": _spread(rng, 8, 128, 8),
            "l": _spread(rng, 1, 64), "requests": m if rng.random() < 0.5 else _spread(rng, 1, min(m, 64)),
            "type": rng.choice(["bf16", "f32"])}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    state = {"case": case}
    if case["op"] == "norm":
        rows, k, t = case["rows"], case["k"], TYPES[case["type"]]
        # Activations: tokens of different magnitude, and a few channels far above the others.
        x = normal(rows, k) * (normal(rows, 1) * 0.5).exp() * (1 + 20 * (uniform(k) < 0.004))
        state |= {"x": x.to(t), "w": (1 + 0.2 * normal(k)).to(t)}
        if case["residual"]:
            state["r"] = (normal(rows, k) * 2).to(t)
        if case["train"]:
            state["dy"] = (normal(rows, k) * 0.01).to(t)
            if case["residual"]:
                state["dh"] = (normal(rows, k) * 0.01).to(t)
    elif case["op"] == "loss":
        m, v, k = case["m"], case["v"], case["k"]
        # Logits of about unit size but for the wanted token's, which the model knows by 0 to 12 more.
        w = (normal(v, k) / math.sqrt(k)).bfloat16()
        target = torch.randint(0, v, (m,), generator=g, device=DEV)
        x = normal(m, k) + 12 * uniform(m, 1) * w[target].float()
        # Whole stretches of tokens without a loss, as prompts are.
        stretch = -(-m // 16)
        none = (uniform(16) < case["ignored"]).repeat_interleave(stretch)[:m]
        target = torch.where(none, torch.full_like(target, IGNORE), target)
        state |= {"x": x.bfloat16(), "w": w, "target": target}
        if case["train"]:
            # The mean's gradient, tokens weighted by their sequences.
            state["dl"] = (0.5 + uniform(m)) / m
    else:
        m, n, k, r, l = (case[i] for i in "mnkrl")
        # The requests' tokens lie one request after the other; a tenth of the requests has no adapter.
        of = torch.randint(0, l, (case["requests"],), generator=g, device=DEV, dtype=torch.int32)
        of = torch.where(uniform(case["requests"]) < 0.1, torch.full_like(of, -1), of)
        if case["requests"] < m:
            starts = torch.randint(0, m, (case["requests"],), generator=g, device=DEV)
            place = (torch.arange(m, device=DEV)[:, None] >= starts).sum(1) % case["requests"]
        else:
            place = torch.arange(m, device=DEV)
        state |= {"x": normal(m, k).bfloat16(), "a": (normal(l, r, k) / math.sqrt(k)).bfloat16(),
                  "b": (0.5 * normal(l, n, r) / math.sqrt(r)).bfloat16(), "index": of[place].contiguous(),
                  "s": 0.5 + 1.5 * uniform(l), "base": normal(m, n).to(TYPES[case["type"]])}
    return state


def _norm(s, case):
    t = s["x"].dtype
    h = s["x"].float() + s["r"].float() if case["residual"] else s["x"].float()
    h = h.to(t).float()
    # The mean in 64 bits: a code next to a border goes by the last bit of the scale.
    inv = (1 / (h.double().square().mean(dim=1, keepdim=True) + EPS).sqrt()).float()
    n, w = h * inv, s["w"].float()
    y = n * w
    if case["out"] != "same":
        most = y.abs().amax(dim=1, keepdim=True)
        scale = most / torch.full_like(most, TOP[case["out"]])
        inverse = (torch.ones_like(scale) / scale).clamp(max=torch.finfo(torch.float32).max)
        q = y * inverse
        if case["out"] == "int8":
            codes = q.round().clamp(-127, 127)
        else:
            # e4m3: 3 bits after the first, the smallest step 2^-9.
            q = q.clamp(-448, 448)
            step = torch.exp2((torch.frexp(q)[1] - 4).clamp(min=-9).float())
            codes = (q / step).round() * step
        return {"values": codes * scale, "scale": scale[:, 0], "h": h.to(t)}
    out = {"y": y.to(t)}
    if case["residual"]:
        out["h"] = h.to(t)
    if case["train"]:
        dy = s["dy"].float()
        gr = dy * w
        dx = inv * (gr - n * (gr * n).mean(dim=1, keepdim=True))
        out |= {"dx": (dx + s["dh"].float() if case["residual"] else dx).to(t), "dw": (dy * n).sum(dim=0).to(t)}
    return out


def _loss(s, case):
    x, w, target = s["x"].float(), s["w"].float(), s["target"]
    some = target != IGNORE
    rows, t = torch.arange(case["m"], device=DEV), target.clamp(min=0)
    z = x @ w.t()
    wanted = z[rows, t]
    top = z.amax(dim=1, keepdim=True)
    p = torch.exp(z - top)
    total = p.sum(dim=1, keepdim=True)
    loss = torch.where(some, top[:, 0] + torch.log(total[:, 0]) - wanted, torch.zeros_like(wanted))
    if not case["train"]:
        return loss
    p = p / total
    p[rows, t] -= 1
    p = p * torch.where(some, s["dl"], torch.zeros_like(s["dl"]))[:, None]
    return {"loss": loss, "dx": (p @ w).bfloat16(), "dw": (p.t() @ x).bfloat16()}


def _adapters(s, case):
    m, n, k, r, l = (case[i] for i in "mnkrl")
    index, a, b = s["index"].long(), s["a"].float(), s["b"].float()
    # The first products of all adapters, of which each row keeps its own one's.
    v = (s["x"].float() @ a.reshape(l * r, k).t()).reshape(m, l, r)
    own_one = index[:, None] == torch.arange(l, device=DEV)
    v = torch.where(own_one[:, :, None], v * s["s"][:, None], torch.zeros_like(v)).reshape(m, l * r)
    return (s["base"].float() + v @ b.transpose(1, 2).reshape(l * r, n)).to(s["base"].dtype)


def _plain(s, case):
    return {"norm": _norm, "loss": _loss, "adapters": _adapters}[case["op"]](s, case)


def _own(s, case):
    import block_scaled_precision_e2m1_amd as fp4

    if case["op"] == "norm":
        if case["out"] != "same":
            r = fp4.rms_norm_quantize(s["x"], s["w"], eps=EPS, residual=s.get("r"), codes=case["out"])
            codes = r[0] if case["out"] == "int8" else r[0].view(torch.float8_e4m3fn).float()
            return {"values": codes * r[1][:, None], "scale": r[1], "h": r[2] if case["residual"] else s["x"]}
        if not case["residual"]:
            y, h = fp4.rms_norm(s["x"], s["w"], eps=EPS), s["x"]
            out = {"y": y}
        else:
            y, h = fp4.rms_norm(s["x"], s["w"], eps=EPS, residual=s["r"])
            out = {"y": y, "h": h}
        if case["train"]:
            out["dx"], out["dw"] = fp4.rms_norm_backward(s["dy"], h, s["w"], eps=EPS, dH=s.get("dh"))
        return out
    if case["op"] == "loss":
        if not case["train"]:
            return fp4.cross_entropy_gemm(s["x"], s["w"], s["target"], ignore_index=IGNORE)
        loss, lse = fp4.cross_entropy_gemm(s["x"], s["w"], s["target"], ignore_index=IGNORE, save=True)
        dx, dw = fp4.cross_entropy_gemm_backward(s["dl"], s["x"], s["w"], s["target"], lse, ignore_index=IGNORE)
        return {"loss": loss, "dx": dx, "dw": dw}
    return fp4.adapter_gemm(s["base"], s["x"], s["a"], s["b"], s["index"], scales=s["s"])


def run(state):
    return _own(state, state["case"]) if own else _plain(state, state["case"])


def work(case):
    if case["op"] == "norm":
        rows, k, e = case["rows"], case["k"], 2 if case["type"] == "bf16" else 4
        # x, the residual and the weight read; the sum and the results (codes and scales) written.
        each = e * (3 if case["residual"] else 1) + (e if case["out"] == "same" else 1)
        total = {"bytes": rows * k * each + k * e + (0 if case["out"] == "same" else 4 * rows), "flops": 4 * rows * k}
        if case["train"]:
            # The incoming gradients read, dx and dw written.
            total["bytes"] += rows * k * e * (3 if case["residual"] else 2) + k * e
            total["flops"] += 8 * rows * k
        return total
    if case["op"] == "loss":
        m, v, k = case["m"], case["v"], case["k"]
        some = m * (1 - case["ignored"])
        total = {"bytes": int(2 * (some * k + v * k) + 12 * m), "flops": int(2 * some * v * k)}
        if case["train"]:
            total["bytes"] += 2 * (m * k + v * k) + 4 * m
            total["flops"] *= 3
        return total
    m, n, k, r, used = case["m"], case["n"], case["k"], case["r"], min(case["l"], case["requests"])
    return {"bytes": 2 * m * k + 2 * m * n * (2 if case["type"] == "bf16" else 4) + used * (2 * r * (k + n) + 4) + 4 * m,
            "flops": 2 * m * r * (k + n)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        t = s["x"].dtype
        x, w = s["x"].double(), s["w"].double().requires_grad_(case["train"])
        if case["residual"]:
            x = torch.add(x, s["r"].double())
        # What is kept of the sum is rounded to the rows' type, and the norm is that of the kept one.
        h = x.to(t).double().requires_grad_(case["train"])
        size = (torch.linalg.vector_norm(h, dim=1, keepdim=True).pow(2) / case["k"] + EPS).sqrt()
        if case["out"] == "same":
            y = h / size * w
            out = {"y": y.detach()} | ({"h": x} if case["residual"] else {})
            if case["train"]:
                dx, dw = torch.autograd.grad(y, (h, w), s["dy"].double())
                out |= {"dx": dx + s["dh"].double() if case["residual"] else dx, "dw": dw}
            return out
        # The definition rounds the inverse size, both products, the scale, its inverse and the scaled value to 32
        # bits: each is formed in 64 here and rounded.
        y = torch.mul(h, size.reciprocal().float().double()).float().double()
        y = torch.mul(y, w).float().double()
        scale = (y.abs().max(dim=1, keepdim=True).values / TOP[case["out"]]).float().double()
        q = torch.mul(y, scale.reciprocal().float().double()).float()
        codes = q.round() if case["out"] == "int8" else q.clamp(-448, 448).to(torch.float8_e4m3fn)
        return {"values": torch.mul(codes.double(), scale), "scale": scale.squeeze(1), "h": x}
    if case["op"] == "loss":
        train = case["train"]
        x, w = (s[i].double().requires_grad_(train) for i in ("x", "w"))
        loss = torch.nn.functional.cross_entropy(torch.mm(x, w.T), s["target"], reduction="none", ignore_index=IGNORE)
        if not train:
            return loss
        dx, dw = torch.autograd.grad(loss, (x, w), s["dl"].double())
        return {"loss": loss.detach(), "dx": dx, "dw": dw}
    y = s["base"].double()
    for i in range(case["l"]):
        at = torch.nonzero(s["index"] == i).squeeze(1)
        if at.numel():
            low = torch.mm(s["x"][at].double(), s["a"][i].double().T)
            y[at] += torch.mm(low, s["b"][i].double().T) * s["s"][i].double()
    return y
