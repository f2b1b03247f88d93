"""Plain 64-bit forms of the operators on 4-bit weights, the packed form read back
by the formulas of include/tw.h, and the bounds their tests use."""
import numpy as np
import torch

LEVELS = {"int4": np.arange(8.0), "e2m1": np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6.0])}
TOP = {"int4": 7.0, "e2m1": 6.0}
TINY = 2.0 ** -117
U = 2.0 ** -24  # half a step of fp32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def bf16(v):
    """float64 values rounded to bf16 (8 bits) once, to nearest even; in range."""
    m, e = np.frexp(v)
    return np.ldexp(np.round(m * 256) / 256, e)


def quantise(w, group, kind):
    """(values [n, k], scales [n, groups]) of float64 weights, by comparison with the
    middles between neighbouring levels; a middle goes to the even code."""
    n, k = w.shape
    levels, top = LEVELS[kind], TOP[kind]
    groups = -(-k // group)
    q, s = np.zeros((n, k)), np.zeros((n, groups))
    for g in range(groups):
        cols = slice(g * group, min(k, (g + 1) * group))
        v = w[:, cols]
        with np.errstate(invalid="ignore"):
            most = np.abs(v).max(axis=1)
        finite = np.isfinite(v).all(axis=1)
        live = finite & (most >= TINY)
        s[:, g] = np.where(live, bf16(np.where(live, most, 1.0) / top),
                           np.where(finite, 0.0, np.nan))
        a = np.abs(v[live])
        scale = s[live, g][:, None]
        code = np.zeros(a.shape, dtype=int)
        for i in range(1, len(levels)):
            middle = (levels[i - 1] + levels[i]) / 2 * scale  # exact: 4 bits times 8
            code += (a >= middle) if i % 2 == 0 else (a > middle)
        out = np.zeros(v.shape)
        out[live] = np.copysign(levels[code], v[live])
        q[:, cols] = out
    return q, s


def unpack(w4):
    """(values [n, k], scales [n, groups], the rest of the codes and scales) of a
    W4Weight."""
    n, k, group = w4.n, w4.k, w4.group
    stripes, tiles = -(-n // 16), -(-k // 128)
    tile_bytes = 1024 + 4096 // group
    raw = w4.packed.cpu().numpy()
    assert raw.size == stripes * tiles * tile_bytes
    raw = raw.reshape(stripes, tiles, tile_bytes)
    rows, cols = np.arange(stripes * 16), np.arange(tiles * 128)
    r, c = rows[:, None] % 16, cols[None, :] % 128
    st, ti = rows[:, None] // 16, cols[None, :] // 128
    at = r // 8 * 512 + (r % 8 * 4 + c // 8 % 4) * 16 + c // 32 * 4
    word = sum(raw[st, ti, at + b].astype(np.uint64) << np.uint64(8 * b) for b in range(4))
    i = c % 8
    half = (word >> (16 * (i % 2)).astype(np.uint64)) & np.uint64(0xffff)
    v = i // 2 + 0 * r
    if w4.kind == "int4":
        values = (half >> (4 * v).astype(np.uint64) & np.uint64(15)).astype(float) - 8
    else:
        sign = half >> np.array([15, 12, 14, 13], dtype=np.uint64)[v] & np.uint64(1)
        code = half >> np.array([6, 3, 9, 0], dtype=np.uint64)[v] & np.uint64(7)
        values = np.where(sign == 1, -1.0, 1.0) * LEVELS["e2m1"][code.astype(int)]
    sat = 1024 + r % 8 * (512 // group) + c // group * 4 + r // 8 * 2
    bits = raw[st, ti, sat].astype(np.uint32) | raw[st, ti, sat + 1].astype(np.uint32) << 8
    scale = (bits << 16).astype(np.uint32).view(np.float32).astype(np.float64)
    # One scale per group.
    per_group = scale[:, ::group]
    assert np.array_equal(per_group.repeat(group, axis=1), scale, equal_nan=True)
    groups = -(-k // group)
    rest = np.concatenate([values[n:].ravel(), values[:, k:].ravel(), per_group[n:].ravel(),
                           per_group[:, groups:].ravel()])
    return values[:n, :k], per_group[:n, :groups], rest


def weights(values, scales, group):
    return values * scales.repeat(group, axis=1)[:, :values.shape[1]]


def product_bound(x, w, out, group, dtype, fp32_x):
    """Error allowed of out = x w^T (64-bit, scales included).  A group's products
    are exact; its sum is a chain of group / 16 matrix steps, each off by a rounding
    or truncation of the sum so far and by the alignment of its 16 terms (8 more of
    them in all); groups, pieces of K (of a tile at least) and the three terms of fp32 x (the
    small ones first) are joined by fp32 additions; a scale multiplies; the result is
    rounded to dtype."""
    size = np.abs(x) @ np.abs(w).T * (1.01 if fp32_x else 1.0)
    tiles = -(-w.shape[1] // 128)
    adds = tiles * (128 // group) + 24 * (3 if fp32_x else 1) + 2
    return half_step(dtype) * np.abs(out) + ((group / 16 + 8) * 2 + adds) * U * size
