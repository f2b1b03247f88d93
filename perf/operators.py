"""The 8-bit operators of a tensor-parallel layer as a benchmark: their cases,
their plain forms and the framework's calls.

  norm      sum of the rank partials + residual, RMS norm, output in 8 bits
            with one scale per token (what the next linear layer reads)
  quantize  rows to 8 bits with one scale per token (the input of a linear
            layer that does not come from a norm: attention, activation)
  product   out[t, n] = xs[t] * ws[n] * sum_k x[t, k] * w[n, k] on 8-bit x, w

8 bits are int8 (values to +-127) or e4m3 (to +-448).  Quantised outputs are
returned as the values they stand for, rounded to bf16, next to their scales.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
QUANT = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}
EPS = 1e-5


def listed():
    return [
        # One decode step of one sequence, eight ranks, 8192 features.
        {"name": "norm_t1_int8", "op": "norm", "parts": 8, "tokens": 1, "hidden": 8192,
         "type": "bf16", "quant": "int8", "outs": 1},
        # A decode batch of 64 sequences.
        {"name": "norm_t64_e4m3", "op": "norm", "parts": 8, "tokens": 64, "hidden": 8192,
         "type": "bf16", "quant": "e4m3", "outs": 1},
        # A prefill chunk of about a thousand tokens over eight ranks.
        {"name": "norm_t1024_int8", "op": "norm", "parts": 8, "tokens": 1024, "hidden": 8192,
         "type": "bf16", "quant": "int8", "outs": 1},
        # The same over two ranks with shorter rows.
        {"name": "norm_t2048_tp2_e4m3", "op": "norm", "parts": 2, "tokens": 2048,
         "hidden": 4096, "type": "bf16", "quant": "e4m3", "outs": 1},
        # fp32 activations, a ragged batch, two gather destinations.
        {"name": "norm_t1111_f32_int8", "op": "norm", "parts": 4, "tokens": 1111,
         "hidden": 5120, "type": "f32", "quant": "int8", "outs": 2},
        # A ragged decode batch with a short odd row.
        {"name": "quantize_t37_h1000_int8", "op": "quantize", "tokens": 37, "hidden": 1000,
         "type": "bf16", "quant": "int8"},
        # The attention output of a prefill chunk.
        {"name": "quantize_t4096_e4m3", "op": "quantize", "tokens": 4096, "hidden": 8192,
         "type": "bf16", "quant": "e4m3"},
        # One token through a square projection: the weights are read once.
        {"name": "product_t1_int8", "op": "product", "tokens": 1, "inner": 8192,
         "channels": 8192, "type": "bf16", "quant": "int8"},
        # A decode batch through one rank's share of a row-parallel layer.
        {"name": "product_t24_k1024_e4m3", "op": "product", "tokens": 24, "inner": 1024,
         "channels": 8192, "type": "bf16", "quant": "e4m3"},
        # A ragged chunk, a channel count off every tile, fp32 partials.
        {"name": "product_t333_f32_int8", "op": "product", "tokens": 333, "inner": 5120,
         "channels": 4090, "type": "f32", "quant": "int8"},
        # A prefill chunk in int8.
        {"name": "product_t1024_int8", "op": "product", "tokens": 1024, "inner": 8192,
         "channels": 8192, "type": "bf16", "quant": "int8"},
        # A long prefill chunk in e4m3.
        {"name": "product_t4096_e4m3", "op": "product", "tokens": 4096, "inner": 8192,
         "channels": 8192, "type": "bf16", "quant": "e4m3"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over their logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "product"])
    case = {"op": op, "type": rng.choice(["bf16", "bf16", "f32"]),
            "quant": rng.choice(["int8", "e4m3"]), "tokens": _spread(rng, 1, 4096)}
    step = 8 if case["type"] == "bf16" else 4  # rows are whole 16-byte vectors
    if op == "product":
        case["inner"] = 16 * _spread(rng, 4, 512)
        case["channels"] = _spread(rng, 64, 8192)
        return case
    case["hidden"] = step * _spread(rng, 64 // step, 8192 // step)
    if op == "norm":
        case["parts"] = rng.randint(1, 8)
        case["outs"] = rng.randint(1, 2)
        most = 8192 * 1024 * 10  # values moved by the largest listed norm
        case["tokens"] = min(case["tokens"],
                             max(1, most // (case["hidden"] * (case["parts"] + 3))))
    return case


def _to_8_bits(x, quant):
    """Rows of x in 8 bits and their scales (a row of zeros: scale 0)."""
    kind, top = QUANT[quant]
    scale = x.abs().amax(-1, keepdim=True) / top
    q = torch.where(scale > 0, x / scale, torch.zeros_like(x)).clamp(-top, top)
    return (q.round() if quant == "int8" else q).to(kind), scale[..., 0]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    kind, t = TYPES[case["type"]], case["tokens"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    def empty(rows, columns, kind):
        return torch.empty(rows, columns, device="cuda", dtype=kind)

    state = {"case": case}
    if case["op"] == "product":
        k, n = case["inner"], case["channels"]
        state["x"], state["x_scale"] = _to_8_bits(normal(t, k), case["quant"])
        state["w"], state["w_scale"] = _to_8_bits(normal(n, k) / math.sqrt(k), case["quant"])
        state["out"] = empty(t, n, kind)
        return state
    h, outs = case["hidden"], case.get("outs", 1)
    if case["op"] == "norm":
        deviation = 1.0 / math.sqrt(case["parts"])
        state["partials"] = [(normal(t, h) * deviation).to(kind) for _ in range(case["parts"])]
        state["residual"] = normal(t, h).to(kind)
        state["weight"] = (torch.rand(h, generator=g, device="cuda") + 0.5).to(kind)
        state["residual_out"] = empty(t, h, kind)
    else:
        state["x"] = normal(t, h).to(kind)
    state["out"] = [empty(t, h, QUANT[case["quant"]][0]) for _ in range(outs)]
    state["scale"] = [torch.empty(t, device="cuda", dtype=torch.float32) for _ in range(outs)]
    state["values"] = [empty(t, h, torch.bfloat16) for _ in range(outs)]
    return state


def _values(q, scale, into):
    """What 8-bit rows stand for: multiplied in 32 bits, rounded to bf16 once."""
    q = q if q.dtype == torch.int8 else q.to(torch.bfloat16)  # e4m3 is exact in bf16
    return torch.mul(q, scale[:, None], out=into)


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "product":
        out = state["x"].float() @ state["w"].float().t()
        return (out * state["x_scale"][:, None] * state["w_scale"]).to(state["out"].dtype)
    if case["op"] == "quantize":
        q, scale = _to_8_bits(state["x"].float(), case["quant"])
        return {"out": _values(q, scale, state["values"][0]), "scale": scale}
    x = torch.stack(state["partials"]).sum(0, dtype=torch.float32) + state["residual"].float()
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * state["weight"].float()
    q, scale = _to_8_bits(y, case["quant"])
    # Every gather destination holds the same rows.
    values = [_values(q, scale, v) for v in state["values"]]
    return {"out": values, "scale": [scale for _ in values],
            "residual": x.to(state["residual"].dtype)}


def _run_own(state, case):
    from reduce_residual_rmsnorm_tw_gb300 import tw
    if case["op"] == "product":
        tw.tw_gemm_q8(state["x"], state["x_scale"], state["w"], state["w_scale"], state["out"])
        return state["out"]
    if case["op"] == "quantize":
        tw.tw_quantize_rows_q8(state["x"], state["out"][0], state["scale"][0])
        return {"out": _values(state["out"][0], state["scale"][0], state["values"][0]),
                "scale": state["scale"][0]}
    tw.tw_fused_reduce_add_rmsnorm_q8(state["partials"], state["residual"], state["weight"],
                                      state["out"], state["scale"], state["residual_out"], EPS)
    return {"out": [_values(q, s, v) for q, s, v in zip(state["out"], state["scale"],
                                                        state["values"])],
            "scale": state["scale"], "residual": state["residual_out"]}


def work(case):
    size, t = (2 if case["type"] == "bf16" else 4), case["tokens"]
    if case["op"] == "product":
        k, n = case["inner"], case["channels"]
        return {"bytes": t * k + n * k + 4 * (t + n) + t * n * size, "flops": 2 * t * n * k}
    h, outs = case["hidden"], case.get("outs", 1)
    quantised = outs * t * (h + 4)
    if case["op"] == "quantize":
        return {"bytes": t * h * size + quantised, "flops": 3 * t * h}
    return {"bytes": (case["parts"] + 2) * t * h * size + h * size + quantised,
            "flops": (case["parts"] + 6) * t * h}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "product":
        x = state["x"].float().double() * state["x_scale"].double().unsqueeze(1)
        w = state["w"].float().double() * state["w_scale"].double().unsqueeze(1)
        return torch.einsum("tk,nk->tn", x, w)
    top = QUANT[case["quant"]][1]
    if case["op"] == "quantize":
        y = state["x"].double()
    else:
        x = state["residual"].double()
        for p in state["partials"]:
            x = x + p.double()
        rms = (torch.linalg.vector_norm(x, dim=1) ** 2 / case["hidden"] + EPS) ** 0.5
        y = x * state["weight"].double() / rms.unsqueeze(1)
    step = y.abs().max(dim=1).values / top
    grid = y / step.unsqueeze(1)
    if case["quant"] == "int8":
        grid = torch.round(grid)
    else:
        # e4m3: three mantissa bits, the least exponent -6.
        power = torch.exp2(torch.floor(torch.log2(grid.abs().clamp(min=2.0 ** -6))) - 3)
        grid = torch.round(grid / power) * power
    values = grid * step.unsqueeze(1)
    if case["op"] == "quantize":
        return {"out": values, "scale": step}
    return {"out": [values] * case["outs"], "scale": [step] * case["outs"], "residual": x}
