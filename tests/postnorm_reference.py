"""The step with two norms in plain 64 bits, and how far fp32 may be off it."""
import numpy as np

U = 2.0 ** -24  # half a step of fp32
# Rounded additions on the way to a row's sum of squares: at most 32 in a thread,
# 1 joining its two lanes, 5 in a warp, 8 warps and 8 CTAs, then 3 roundings up to the mean
# plus eps; the reciprocal root is within 2 ulp = 4 U.
SQUARES = 32 + 1 + 5 + 8 + 8 + 3
ROOT = 4 * U


def _rows(v):
    return np.linalg.norm(v, axis=1, keepdims=True)


def step(d, post_weight=None, gate=None, gate_tokens=1, block_scale=1.0, residual_scale=1.0,
         eps=1e-6, post_eps=None):
    """(x, out, error allowed of x, of out), before they are rounded to their type;
    d: partials, residual and weight as float64 arrays."""
    block_scale, residual_scale = float(np.float32(block_scale)), float(np.float32(residual_scale))
    s = sum(d["partials"])
    es = (len(d["partials"]) - 1) * U * sum(np.abs(p) for p in d["partials"])
    u, eu = s, es
    post_eps = float(np.float32(eps if post_eps is None else post_eps))
    eps = float(np.float32(eps))
    if post_weight is not None:
        c = 1 / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + post_eps)
        rel = SQUARES * U / 2 + ROOT + _rows(es) / np.maximum(_rows(s), 1e-300)
        u = s * c * post_weight
        eu = np.abs(u) * (rel + 2 * U) + np.abs(c * post_weight) * es
    if gate is not None:
        g = gate[np.arange(len(s)) // gate_tokens]
        u, eu = u * g, np.abs(g) * eu + U * np.abs(u * g)
    r = residual_scale * d["residual"]
    x = r + block_scale * u
    ex = abs(block_scale) * eu + U * (np.abs(r) + np.abs(x))
    inv = 1 / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps)
    rel = SQUARES * U / 2 + ROOT + _rows(ex) / np.maximum(_rows(x), 1e-300)
    y = x * inv * d["weight"]
    ey = np.abs(y) * (rel + 2 * U) + np.abs(inv * d["weight"]) * ex
    # Terms of second order, and values below fp32's normal range.
    return x, y, ex * 1.01 + 2.0 ** -140, ey * 1.01 + 2.0 ** -140
