"""Plain 64-bit forms of the 8-bit operators and the bounds their tests use.

A quantised row is held as values q with one scale s = max|v| / top.  With
v_t = v / s exact, a correct q differs from v_t by at most half a step of its
type -- 1/2 for int8, eps/2 = 2^-4 of |v_t| for e4m3 (half of its least step
2^-9 below the normal range) -- plus what the fp32 arithmetic before the
rounding is off: top times its relative error.
"""
import numpy as np
import torch

TOP = {"int8": 127.0, "e4m3": 448.0}
KIND = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
U = 2.0 ** -24  # half a step of fp32


def f64(t):
    """Exact widening to a float64 numpy array (8-bit floats included)."""
    t = t.detach()
    if t.dtype == torch.float8_e4m3fn:
        t = t.to(torch.float32)
    return t.cpu().to(torch.float64).numpy()


def row_error(terms, x):
    """Relative error of a row's largest value when each element is an fp32
    sum of len(terms) terms taken in order: (n - 1) roundings of at most
    sum|term|, compared with the row's largest |x|."""
    size = sum(np.abs(t) for t in terms).max(axis=1)
    top = np.abs(x).max(axis=1)
    return (len(terms) - 1) * U * size / np.where(top > 0, top, 1.0)


def check_rows(q, scale, v, quant, rel, what):
    """q [T, H] (8-bit) and scale [T] against the exact rows v, whose fp32
    counterparts are off by at most rel[t] of the row's largest value."""
    g, s = f64(q), f64(scale)
    want = np.abs(v).max(axis=1) / TOP[quant]
    assert np.all(np.abs(s - want) <= rel * want), \
        f"{what}: scale off by {np.max(np.abs(s - want) / want)} relative"
    live = want > 0
    vt = v[live] / want[live, None]
    err = np.abs(g[live] - vt)
    half = np.full_like(vt, 0.5) if quant == "int8" else np.maximum(np.abs(vt) * 2.0 ** -4,
                                                                    2.0 ** -10)
    bound = half + TOP[quant] * rel[live, None]
    bad = err > bound
    assert not bad.any(), f"{what}: {bad.sum()} values off, worst {np.max(err - bound)}"
    assert np.all(g[~live] == 0)


def product(x, x_scale, w, w_scale):
    """(out, size): the product in 64 bits, and sum_k |x w| with the scales."""
    xs, ws = f64(x_scale)[:, None], f64(w_scale)[None, :]
    a, b = f64(x), f64(w)
    return a @ b.T * xs * ws, np.abs(a) @ np.abs(b).T * np.abs(xs * ws)


def product_bound(out, size, raw_size, K, dtype):
    """Error allowed of out[t, n].  The two scale multiplies and the last
    rounding: 3 half steps of fp32, and half a step of bf16 (2^-8) where that
    is the output.  The sum: exact for whole numbers below 2^24; otherwise one
    rounding or truncation (at most 2^-23 of the running sum, itself at most
    sum|x w|) for each of the K / 16 sums that the longest chain can have, and
    for each of the 32 terms inside one."""
    bound = 3 * U * np.abs(out)
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * np.abs(out) * (1 + 3 * U)
    chain = (K / 16 + 32) * 2.0 ** -23 * size
    return bound + np.where(raw_size < 2.0 ** 24, 0.0, chain)


def check_product(out, x, x_scale, w, w_scale, what):
    want, size = product(x, x_scale, w, w_scale)
    if x.dtype == torch.int8:
        raw = np.abs(f64(x)) @ np.abs(f64(w)).T
    else:
        raw = np.full_like(want, np.inf)
    err = np.abs(f64(out) - want)
    bound = product_bound(want, size, raw, x.shape[1], out.dtype)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} elements off; first "
                           f"{tuple(np.argwhere(bad)[0])}, worst ratio "
                           f"{np.nanmax(err / np.maximum(bound, 1e-300))}")


def draw_8_bit(rows, columns, quant, seed, device="cuda"):
    """Random 8-bit rows over the type's whole finite range, and scales."""
    g = torch.Generator()
    g.manual_seed(seed)
    if quant == "int8":
        q = torch.randint(-128, 128, (rows, columns), generator=g, dtype=torch.int32).to(torch.int8)
    else:
        q = (torch.randn(rows, columns, generator=g) * 60).clamp(-448, 448).to(
            torch.float8_e4m3fn)
    s = torch.rand(rows, generator=g) * 0.02 + 0.001
    return q.to(device), s.to(device)
