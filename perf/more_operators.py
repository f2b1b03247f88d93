"""The operators of a layer with sandwich norms and 4-bit weights as a benchmark:
their cases, their plain forms and the framework's calls.

  norm      sum of the rank partials, RMS norm of the block's output, gate and
            scales, residual add, RMS norm of the result:
              s   = sum_r partials[r]
              u   = s / rms(s) * post_weight          (u = s without a post norm)
              x   = residual_scale * residual + block_scale * gate * u
              out = x / rms(x) * weight,   residual_out = x
            out in the inputs' type, or in 8 bits with one scale per token
  product   out[t, n] = xs[t] * sum_k x[t, k] * w[n, k] with w in 4 bits and one
            scale per channel and group of K; x in 16, 32 or 8 bits
  weights   rows of weights to 4 bits with group scales, and read back

4 bits are int4 (values to +-7) or e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives); a group's scale is its largest magnitude / top, rounded to bf16.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
QUANT = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}
TOP4 = {"int4": 7.0, "e2m1": 6.0}
EPS = 1e-5


def listed():
    return [
        # One decode step of one sequence, eight ranks, norms before and after.
        {"name": "norm_t1", "op": "norm", "parts": 8, "tokens": 1, "hidden": 8192,
         "type": "bf16", "quant": "none", "post": True, "gate": "none", "outs": 1,
         "block_scale": 1.0, "residual_scale": 1.0},
        # A decode batch whose next linear layer reads 8 bits.
        {"name": "norm_t64_int8", "op": "norm", "parts": 8, "tokens": 64, "hidden": 8192,
         "type": "bf16", "quant": "int8", "post": True, "gate": "none", "outs": 1,
         "block_scale": 0.22, "residual_scale": 1.0},
        # A prefill chunk of about a thousand tokens over eight ranks.
        {"name": "norm_t1024", "op": "norm", "parts": 8, "tokens": 1024, "hidden": 8192,
         "type": "bf16", "quant": "none", "post": True, "gate": "none", "outs": 1,
         "block_scale": 1.0, "residual_scale": 1.0},
        # Two ranks with shorter rows, every token with a gate of its own (gated output).
        {"name": "norm_t2048_tp2_gated", "op": "norm", "parts": 2, "tokens": 2048,
         "hidden": 4096, "type": "bf16", "quant": "none", "post": True, "gate": "token",
         "outs": 1, "block_scale": 1.0, "residual_scale": 1.0},
        # fp32 activations, a gate per sequence of 300 tokens (a conditioned block), no
        # post norm, a scaled residual, two gather destinations.
        {"name": "norm_t1111_f32_conditioned", "op": "norm", "parts": 4, "tokens": 1111,
         "hidden": 5120, "type": "f32", "quant": "none", "post": False, "gate": "sequence",
         "outs": 2, "block_scale": 1.0, "residual_scale": 1.414},
        # One token through a square projection: the weights are read once.
        {"name": "product_t1_int4", "op": "product", "tokens": 1, "inner": 8192,
         "channels": 8192, "group": 128, "kind": "int4", "x": "bf16", "out": "bf16"},
        # One token through one rank's share of a row-parallel layer, fine groups.
        {"name": "product_t1_k1024_e2m1", "op": "product", "tokens": 1, "inner": 1024,
         "channels": 8192, "group": 32, "kind": "e2m1", "x": "bf16", "out": "bf16"},
        # A few fp32 tokens (a draft's tokens being checked), fp32 partials.
        {"name": "product_t5_f32", "op": "product", "tokens": 5, "inner": 4096,
         "channels": 5120, "group": 64, "kind": "int4", "x": "f32", "out": "f32"},
        # A decode batch in 8 bits, as the norm hands it over; a channel count off every
        # tile.
        {"name": "product_t16_int8", "op": "product", "tokens": 16, "inner": 5120,
         "channels": 4090, "group": 128, "kind": "int4", "x": "int8", "out": "bf16"},
        # A decode batch through the widest layer.
        {"name": "product_t8_n32768_int4", "op": "product", "tokens": 8, "inner": 8192,
         "channels": 32768, "group": 128, "kind": "int4", "x": "bf16", "out": "bf16"},
        # A projection's weights laid out once in 4 bits, and read back for a long prompt.
        {"name": "weights_8192_int4", "op": "weights", "inner": 8192, "channels": 8192,
         "group": 128, "kind": "int4", "type": "bf16"},
        # fp32 weights, fine groups, a channel count off every tile.
        {"name": "weights_4090_f32_e2m1", "op": "weights", "inner": 5120, "channels": 4090,
         "group": 32, "kind": "e2m1", "type": "f32"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over their logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "product", "weights"])
    if op == "norm":
        case = {"op": op, "type": rng.choice(["bf16", "bf16", "f32"]),
                "quant": rng.choice(["none", "none", "int8", "e4m3"]),
                "post": rng.random() < 0.75, "gate": rng.choice(["none", "token", "sequence"]),
                "parts": rng.randint(1, 8), "outs": rng.randint(1, 2),
                "block_scale": rng.choice([1.0, 0.22, 0.5]),
                "residual_scale": rng.choice([1.0, 1.0, 1.414])}
        step = 8 if case["type"] == "bf16" else 4  # rows are whole 16-byte vectors
        case["hidden"] = step * _spread(rng, 64 // step, 8192 // step)
        most = 8192 * 1024 * 10  # values moved by the largest listed norm
        case["tokens"] = min(_spread(rng, 1, 4096),
                             max(1, most // (case["hidden"] * (case["parts"] + 4))))
        return case
    case = {"op": op, "group": rng.choice([32, 64, 128]), "kind": rng.choice(["int4", "e2m1"]),
            "inner": 16 * _spread(rng, 4, 512)}
    if op == "weights":
        case["channels"] = _spread(rng, 16, 8192)
        case["type"] = rng.choice(["bf16", "f32"])
        return case
    case["channels"] = _spread(rng, 64, 32768)
    case["tokens"] = _spread(rng, 1, 16)
    case["x"] = rng.choice(["bf16", "bf16", "f32", "int8", "e4m3"])
    case["out"] = rng.choice(["bf16", "f32"])
    return case


def _to_8_bits(x, quant):
    """Rows of x in 8 bits and their scales (a row of zeros: scale 0)."""
    kind, top = QUANT[quant]
    scale = x.abs().amax(-1, keepdim=True) / top
    q = torch.where(scale > 0, x / scale, torch.zeros_like(x)).clamp(-top, top)
    return (q.round() if quant == "int8" else q).to(kind), scale[..., 0]


def _to_4_bits(w, group, kind):
    """Rows of w as 4-bit values (float32, on the type's grid) and the bf16 scales of
    their groups, as float32 [N, groups].  In 64 bits: many quotients are ties."""
    n, k = w.shape
    top = TOP4[kind]
    groups = -(-k // group)
    v = torch.zeros(n, groups * group, device=w.device, dtype=torch.float64)
    v[:, :k] = w
    v = v.view(n, groups, group)
    mantissa, exponent = torch.frexp(v.abs().amax(-1) / top)
    scale = torch.ldexp(torch.round(mantissa * 256) / 256, exponent)  # bf16: 8 bits
    q = torch.where(scale[..., None] > 0, v / scale[..., None], torch.zeros_like(v))
    if kind == "int4":
        q = q.round()
    else:
        a = q.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
        q = torch.copysign((a / step).round() * step, q)
    q = q.clamp(-top, top).view(n, -1)[:, :k]
    return q.float().contiguous(), scale.float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    state = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    def uniform(n):
        return torch.rand(n, generator=g, device="cuda") + 0.5

    def empty(rows, columns, kind):
        return torch.empty(rows, columns, device="cuda", dtype=kind)

    if case["op"] == "norm":
        t, h, kind = case["tokens"], case["hidden"], TYPES[case["type"]]
        deviation = 1.0 / math.sqrt(case["parts"])
        state["partials"] = [(normal(t, h) * deviation).to(kind) for _ in range(case["parts"])]
        state["residual"] = normal(t, h).to(kind)
        state["weight"] = uniform(h).to(kind)
        state["post_weight"] = uniform(h).to(kind) if case["post"] else None
        # Tokens that share a row of the gate.
        state["gate_tokens"] = {"none": 1, "token": 1, "sequence": 300}[case["gate"]]
        rows = -(-t // state["gate_tokens"])
        state["gate"] = None if case["gate"] == "none" else (0.5 * normal(rows, h)).to(kind)
        state["residual_out"] = empty(t, h, kind)
        if case["quant"] == "none":
            state["out"] = [empty(t, h, kind) for _ in range(case["outs"])]
        else:
            state["out"] = [empty(t, h, QUANT[case["quant"]][0]) for _ in range(case["outs"])]
            state["scale"] = [torch.empty(t, device="cuda") for _ in range(case["outs"])]
            state["values"] = [empty(t, h, torch.bfloat16) for _ in range(case["outs"])]
        return state
    n, k = case["channels"], case["inner"]
    w = normal(n, k) / math.sqrt(k)
    if case["op"] == "weights":
        state["w"] = w.to(TYPES[case["type"]])
        state["values"] = empty(n, k, TYPES[case["type"]])
        if own:
            from reduce_residual_rmsnorm_tw_gb300 import tw
            state["w4"] = tw.W4Weight(n, k, case["group"], case["kind"])
        return state
    q, scale = _to_4_bits(w, case["group"], case["kind"])
    state["q"] = q.to(torch.bfloat16)  # exact
    state["q_scale"] = scale
    if own:
        # What a loader does with a checkpoint's codes and scales, once.
        from reduce_residual_rmsnorm_tw_gb300 import tw
        state["w4"] = tw.W4Weight.from_values(state["q"], scale, case["group"], case["kind"])
    x = normal(case["tokens"], k)
    state["x_scale"] = None
    if case["x"] in QUANT:
        state["x"], state["x_scale"] = _to_8_bits(x, case["x"])
    else:
        state["x"] = x.to(TYPES[case["x"]])
    state["out"] = empty(case["tokens"], n, TYPES[case["out"]])
    return state


def _values(q, scale, into):
    """What 8-bit rows stand for: multiplied in 32 bits, rounded to bf16 once."""
    q = q if q.dtype == torch.int8 else q.to(torch.bfloat16)  # e4m3 is exact in bf16
    return torch.mul(q, scale[:, None], out=into)


def _spread_scale(scale, group, k):
    """One scale per value."""
    return scale.repeat_interleave(group, dim=1)[:, :k]


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "product":
        w = state["q"].float() * _spread_scale(state["q_scale"], case["group"], case["inner"])
        out = state["x"].float() @ w.t()
        if state["x_scale"] is not None:
            out = out * state["x_scale"][:, None]
        return out.to(state["out"].dtype)
    if case["op"] == "weights":
        q, scale = _to_4_bits(state["w"], case["group"], case["kind"])
        return (q * _spread_scale(scale, case["group"], case["inner"])).to(state["w"].dtype)
    u = torch.stack(state["partials"]).sum(0, dtype=torch.float32)
    if state["post_weight"] is not None:
        u = u / torch.sqrt(u.square().mean(-1, keepdim=True) + EPS) * state["post_weight"].float()
    if state["gate"] is not None:
        rows = torch.arange(u.shape[0], device=u.device) // state["gate_tokens"]
        u = u * state["gate"].float()[rows]
    x = case["residual_scale"] * state["residual"].float() + case["block_scale"] * u
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * state["weight"].float()
    residual = x.to(state["residual"].dtype)
    # Every gather destination holds the same rows.
    if case["quant"] == "none":
        return {"out": [o.copy_(y) for o in state["out"]], "residual": residual}
    q, scale = _to_8_bits(y, case["quant"])
    return {"out": [_values(q, scale, v) for v in state["values"]],
            "scale": [scale for _ in state["values"]], "residual": residual}


def _run_own(state, case):
    from reduce_residual_rmsnorm_tw_gb300 import tw
    if case["op"] == "product":
        tw.tw_gemm_w4(state["x"], state["w4"], state["out"], x_scale=state["x_scale"])
        return state["out"]
    if case["op"] == "weights":
        tw.tw_quantize_w4(state["w"], state["w4"])
        tw.tw_dequantize_w4(state["w4"], state["values"])
        return state["values"]
    block = {"post_weight": state["post_weight"], "gate": state["gate"],
             "gate_tokens": state["gate_tokens"], "block_scale": case["block_scale"],
             "residual_scale": case["residual_scale"]}
    if case["quant"] == "none":
        tw.tw_fused_reduce_postnorm_add_rmsnorm(
            state["partials"], state["residual"], state["weight"], state["out"],
            state["residual_out"], EPS, **block)
        return {"out": state["out"], "residual": state["residual_out"]}
    tw.tw_fused_reduce_postnorm_add_rmsnorm_q8(
        state["partials"], state["residual"], state["weight"], state["out"], state["scale"],
        state["residual_out"], EPS, **block)
    return {"out": [_values(q, s, v) for q, s, v in zip(state["out"], state["scale"],
                                                        state["values"])],
            "scale": state["scale"], "residual": state["residual_out"]}


def work(case):
    if case["op"] == "norm":
        size, t, h = (2 if case["type"] == "bf16" else 4), case["tokens"], case["hidden"]
        gate = {"none": 0, "token": t, "sequence": -(-t // 300)}[case["gate"]]
        out = t * h * size if case["quant"] == "none" else t * (h + 4)
        rows = (case["parts"] + 2) * t + gate + 1 + (1 if case["post"] else 0)
        return {"bytes": rows * h * size + case["outs"] * out,
                "flops": (case["parts"] + 12) * t * h}
    n, k = case["channels"], case["inner"]
    packed = n * k // 2 + 2 * n * -(-k // case["group"])
    if case["op"] == "weights":
        size = 2 if case["type"] == "bf16" else 4
        return {"bytes": 2 * n * k * size + packed, "flops": 4 * n * k}
    t = case["tokens"]
    x = t * k * {"bf16": 2, "f32": 4}.get(case["x"], 1) + (4 * t if case["x"] in QUANT else 0)
    return {"bytes": packed + x + t * n * (2 if case["out"] == "bf16" else 4),
            "flops": 2 * t * n * k}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "product":
        x = state["x"].float().double()
        if state["x_scale"] is not None:
            x = x * state["x_scale"].double().unsqueeze(1)
        column = torch.arange(case["inner"], device=x.device) // case["group"]
        return torch.einsum("tk,nk->tn", x,
                            state["q"].double() * state["q_scale"].double()[:, column])
    if case["op"] == "weights":
        return _exact_weights(state["w"].double(), case)
    s = torch.zeros_like(state["residual"], dtype=torch.float64)
    for p in state["partials"]:
        s += p
    h = case["hidden"]
    if case["post"]:
        s = s * (torch.linalg.vector_norm(s, dim=1, keepdim=True) ** 2 / h + EPS) ** -0.5
        s *= state["post_weight"].double()
    if case["gate"] != "none":
        s *= state["gate"].double().repeat_interleave(state["gate_tokens"], 0)[:len(s)]
    x = state["residual"].double() * case["residual_scale"] + s * case["block_scale"]
    y = x * (torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / h + EPS) ** -0.5
    y *= state["weight"].double()
    if case["quant"] == "none":
        return {"out": [y] * case["outs"], "residual": x}
    step = y.abs().max(dim=1).values / QUANT[case["quant"]][1]
    grid = y / step.unsqueeze(1)
    if case["quant"] == "int8":
        grid = torch.round(grid)
    else:
        # e4m3: three mantissa bits, the least exponent -6.
        power = torch.exp2(torch.floor(torch.log2(grid.abs().clamp(min=2.0 ** -6))) - 3)
        grid = torch.round(grid / power) * power
    return {"out": [grid * step.unsqueeze(1)] * case["outs"], "scale": [step] * case["outs"],
            "residual": x}


def _exact_weights(w, case):
    """Group by group, the nearest of the type's values by comparison with the middles
    between neighbours (a middle itself goes to the one with the even code)."""
    levels = ([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0] if case["kind"] == "e2m1"
              else [float(i) for i in range(8)])
    out = torch.empty_like(w)
    for k in range(0, w.shape[1], case["group"]):
        v = w[:, k:k + case["group"]]
        most = v.abs().max(dim=1, keepdim=True).values
        ratio = most / levels[-1]
        ulp = torch.exp2(torch.floor(torch.log2(ratio.clamp(min=1e-300))) - 7)
        step = torch.round(ratio / ulp) * ulp
        value = torch.zeros_like(v)
        for i in range(1, len(levels)):
            middle = (levels[i - 1] + levels[i]) / 2 * step
            above = v.abs() >= middle if i % 2 == 0 else v.abs() > middle
            value = torch.where(above, levels[i] * step, value)
        out[:, k:k + case["group"]] = torch.where(most > 0, torch.sign(v) * value, 0.0)
    return out
