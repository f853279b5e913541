"""The 8-bit operators of a quantized linear, as cases that can be timed and compared.

Three operators and their use together:

  tokens   quantize_tokens: each row of X to 8-bit codes, q = rint(127 x / max|x|), its scale
           max|x| / 127, the sum of its codes and the values the codes stand for;
  norm     block_norm: r' = r + a g * rms(h) w_post, out = rms(r') w_pre, with the norm after the
           block, its gate g and its scale a, and the norm before the next block;
  product  linear: Y = s_x s_w (sum_k q_x (q_w - z)) + bias from 8-bit tokens and weights;
  norm_product   block_norm whose output is 8-bit tokens, and the product that reads them;
  gate_product   quantize_tokens of silu(gate) * x, and the product that reads them.

`run` computes them in elementary torch operations, or, where `own` is true, by this package's calls.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one new token on its way into a 4096-wide linear
        {"name": "tokens_1x4096", "op": "tokens", "type": "bf16", "m": 1, "k": 4096},
        # a calibration batch at the input of a down projection
        {"name": "tokens_8192x11008", "op": "tokens", "type": "bf16", "m": 8192, "k": 11008},
        # a ragged float32 batch of an odd width
        {"name": "tokens_333x5003_f32", "op": "tokens", "type": "f32", "m": 333, "k": 5003},
        # between two blocks, one new token
        {"name": "norm_1x4096", "op": "norm", "type": "bf16", "m": 1, "k": 4096, "post": True, "gate_rows": 1, "scale": 1.0},
        # between two blocks, a long prompt, one gate row for each of its sequences
        {"name": "norm_16384x4096", "op": "norm", "type": "bf16", "m": 16384, "k": 4096, "post": True, "gate_rows": 2048, "scale": 0.5},
        # an odd width in float16, without the norm after the block and without a gate
        {"name": "norm_1000x5003_f16", "op": "norm", "type": "f16", "m": 1000, "k": 5003, "post": False, "gate_rows": 0, "scale": 1.0},
        # q projection of one new token
        {"name": "product_1x4096x4096", "op": "product", "type": "bf16", "m": 1, "n": 4096, "k": 4096, "zeros": True, "bias": False},
        # up projection of a small decoding batch
        {"name": "product_24x11008x4096", "op": "product", "type": "bf16", "m": 24, "n": 11008, "k": 4096, "zeros": True, "bias": False},
        # down projection of a long prompt
        {"name": "product_8192x4096x11008", "op": "product", "type": "bf16", "m": 8192, "n": 4096, "k": 11008, "zeros": True, "bias": False},
        # odd sizes in every direction, symmetric weights, a bias, float32 out
        {"name": "product_777x1000x1003_f32", "op": "product", "type": "f32", "m": 777, "n": 1000, "k": 1003, "zeros": False, "bias": True},
        # from the residual stream through the norm into an up projection, a prompt
        {"name": "norm_product_2048x11008x4096", "op": "norm_product", "type": "bf16", "m": 2048, "n": 11008, "k": 4096, "post": False, "gate_rows": 0, "scale": 1.0},
        # the gated activation into the down projection, a few new tokens
        {"name": "gate_product_4x4096x11008", "op": "gate_product", "type": "bf16", "m": 4, "n": 4096, "k": 11008},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["tokens", "norm", "product", "product", "norm_product", "gate_product"])
    # where 8-bit codes lie between the input and the output, a value next to a border may take either
    # code, and float32 would show that: those cases have 16-bit types
    kind = rng.choice(["bf16", "bf16", "f16"] + ["f32"] * (op in ("tokens", "norm", "product")))
    m = _log(rng, 1, 8192)
    k = _log(rng, 64, 11008)
    if rng.random() < 0.6:  # widths of models are round, others happen
        k = max(64, k // 64 * 64)
    case = {"op": op, "type": kind, "m": m, "k": k}
    if op in ("norm", "norm_product"):
        case |= {"post": rng.random() < 0.5, "gate_rows": rng.choice([0, 1, 17, m]), "scale": rng.choice([1.0, 0.25])}
    if op in ("product", "norm_product", "gate_product"):
        n = _log(rng, 64, 11008)
        if rng.random() < 0.6:
            n = max(64, n // 64 * 64)
        case["n"] = n
        case["m"] = max(1, min(m, 8192 * 4096 * 11008 // (n * k)))
        if "gate_rows" in case and case["gate_rows"] > case["m"]:
            case["gate_rows"] = case["m"]
    if op == "product":
        case |= {"zeros": rng.random() < 0.7, "bias": rng.random() < 0.3}
    return case


def _pitched(codes):
    """The same 8-bit rows at a pitch of a multiple of 16 bytes, as the products read them."""
    rows, k = codes.shape
    wide = torch.zeros(rows, (k + 15) // 16 * 16, dtype=torch.int8, device=codes.device)
    wide[:, :k] = codes
    return wide[:, :k]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, t, m, k = case["op"], TYPES[case["type"]], case["m"], case["k"]
    state = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def codes(rows, spread):
        return _pitched((normal(rows, k) * spread).round().clamp(-127, 127).to(torch.int8))

    # a few channels are far larger than the others, as activations of decoders have them
    channel = torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, torch.exp(1.5 * normal(k)), torch.ones((), device="cuda"))
    if op in ("tokens", "gate_product"):
        state["x"] = (normal(m, k) * channel).to(t)
    if op == "gate_product":
        state["gate"] = normal(m, k).to(t)
    if op in ("norm", "norm_product"):
        state["h"] = (normal(m, k) * 0.7).to(t)
        state["r"] = (normal(m, k) * channel).to(t)
        state["w_pre"] = 1 + 0.1 * normal(k)
        state["w_post"] = 1 + 0.1 * normal(k) if case["post"] else None
        rows = case["gate_rows"]
        state["gate"] = (1 + 0.2 * normal(-(-m // rows), k)).to(t) if rows else None
    if op in ("product", "norm_product", "gate_product"):
        n = case["n"]
        state["w"] = codes(n, 40.0)
        state["w_scales"] = (0.02 / 40) * (1 + 0.2 * torch.rand(n, generator=g, device="cuda"))
        state["w_zeros"] = torch.randint(-20, 21, (n,), generator=g, device="cuda", dtype=torch.int32) if case.get("zeros", True) else None
        state["bias"] = normal(n) * 0.1 if case.get("bias") else None
    if op == "product":
        state["x"] = codes(m, 30.0)
        state["x_scales"] = (1 / 30) * (1 + torch.rand(m, generator=g, device="cuda"))
        state["x_sums"] = state["x"].sum(1, dtype=torch.int32)
    return state


def _codes(x):
    """(codes, scales) of the rows of x. What lies next to a border between two codes is decided in 64 bits."""
    top = x.abs().amax(1, keepdim=True).double()
    q = torch.round(127.0 * x.double() / torch.where(top > 0, top, torch.ones_like(top)))
    return q.float(), (top / 127.0).float()


def _rms(x):
    return x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)


def _stream(s):
    """The new residual stream, in 32 bits."""
    c = s["case"]
    h = s["h"].float()
    if s["w_post"] is not None:
        h = _rms(h) * s["w_post"]
    if s["gate"] is not None:
        h = h * s["gate"].float().repeat_interleave(c["gate_rows"], 0)[: c["m"]]
    return s["r"].float() + c["scale"] * h


def _product(s, q, scales):
    w = s["w"].float()
    if s["w_zeros"] is not None:
        w = w - s["w_zeros"].float()[:, None]
    y = (q @ w.t()) * s["w_scales"] * scales
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(TYPES[s["case"]["type"]])


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    t = TYPES[c["type"]]
    if c["op"] == "tokens":
        q, scales = _codes(state["x"].float())
        return {"hat": (q * scales).to(t), "scales": scales[:, 0], "sums": q.sum(1, dtype=torch.float64).to(torch.int32)}
    if c["op"] == "norm":
        r = _stream(state)
        return {"stream": r.to(t), "out": (_rms(r) * state["w_pre"]).to(t)}
    if c["op"] == "product":
        return _product(state, state["x"].float(), state["x_scales"][:, None])
    if c["op"] == "norm_product":
        r = _stream(state)
        return {"stream": r.to(t), "y": _product(state, *_codes(_rms(r) * state["w_pre"]))}
    a = state["gate"].float()
    return _product(state, *_codes(a / (1 + torch.exp(-a)) * state["x"].float()))


def _run_own(s):
    from post_weight_quantization_accumulate_b200 import w8a8

    c = s["case"]
    t = TYPES[c["type"]]
    if c["op"] == "tokens":
        x = w8a8.quantize_tokens(s["x"], hat=True)
        return {"hat": x.hat, "scales": x.scales, "sums": x.sums}
    if c["op"] in ("norm", "norm_product"):
        stream, out = w8a8.block_norm(s["h"], s["r"], s["w_pre"], post_norm=c["post"], post_weight=s["w_post"], gate=s["gate"],
                                      gate_rows=c["gate_rows"], scale=c["scale"], eps=EPS, quantize=c["op"] == "norm_product")
        if c["op"] == "norm":
            return {"stream": stream, "out": out}
    if c["op"] == "product":
        out = w8a8.Tokens(s["x"], s["x_scales"], s["x_sums"])
    elif c["op"] == "gate_product":
        out = w8a8.quantize_tokens(s["x"], gate=s["gate"])
    y = w8a8.linear(out, w8a8.Weight(s["w"], s["w_scales"], s["w_zeros"]), bias=s["bias"], dtype=t)
    return {"stream": stream, "y": y} if c["op"] == "norm_product" else y


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    e = 4 if case["type"] == "f32" else 2
    n = case.get("n", 0)
    weights = n * k + 4 * n + (4 * n if case.get("zeros", True) else 0) + (4 * n if case.get("bias") else 0) if n else 0
    gates = -(-m // case["gate_rows"]) * k * e if case.get("gate_rows") else 0
    norm = 2 * m * k * e + gates + 4 * k * (2 if case.get("post") else 1)
    if op == "tokens":  # x in; codes, values, scale and sum out
        return {"bytes": m * k * (2 * e + 1) + 8 * m, "flops": 4 * m * k}
    if op == "norm":  # block, stream, gate and weights in; stream and output out
        return {"bytes": norm + 2 * m * k * e, "flops": 12 * m * k}
    if op == "product":
        return {"bytes": m * k + 8 * m + weights + m * n * e, "flops": 2 * m * n * k}
    if op == "norm_product":
        return {"bytes": norm + m * k * e + weights + m * n * e, "flops": 12 * m * k + 2 * m * n * k}
    return {"bytes": 2 * m * k * e + weights + m * n * e, "flops": 10 * m * k + 2 * m * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64

    def quantized(v):
        top, _ = torch.max(torch.abs(v), dim=-1)
        step = top / 127
        return torch.round(v / torch.where(step == 0, 1.0, step)[:, None]), step

    def normed(v, w):
        return v / torch.sqrt(torch.linalg.vector_norm(v, dim=-1).square() / v.shape[1] + EPS)[:, None] * w.to(f8)[None]

    def times(q, step):
        y = torch.einsum("mk,nk->mn", q, s["w"].to(f8))
        if s["w_zeros"] is not None:
            y = y - torch.outer(q.sum(-1), s["w_zeros"].to(f8))
        y = torch.einsum("mn,m,n->mn", y, step, s["w_scales"].to(f8))
        return y if s["bias"] is None else y + s["bias"].to(f8)

    if case["op"] == "product":
        return times(s["x"].to(f8), s["x_scales"].to(f8))
    if case["op"] == "tokens":
        x = s["x"].to(f8)
        top = x.abs().max(dim=-1).values
        q = torch.round(x * 127 / torch.where(top == 0, 1.0, top)[:, None])
        return {"hat": q * (top / 127)[:, None], "scales": top / 127, "sums": q.sum(-1).to(torch.int32)}
    if case["op"] == "gate_product":
        return times(*quantized(s["gate"].to(f8) * torch.sigmoid(s["gate"].to(f8)) * s["x"].to(f8)))
    h = s["h"].to(f8)
    if s["w_post"] is not None:
        h = normed(h, s["w_post"])
    if s["gate"] is not None:
        rows = torch.arange(case["m"], device="cuda") // case["gate_rows"]
        h = h * s["gate"].to(f8)[rows]
    r = torch.add(s["r"].to(f8), h, alpha=case["scale"])
    out = normed(r, s["w_pre"])
    return {"stream": r, "out": out} if case["op"] == "norm" else {"stream": r, "y": times(*quantized(out))}
