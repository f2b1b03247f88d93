"""check_rows of tests/q8_reference.py for rows that hold finite values only: a
comparison err > bound is false for a NaN code, so codes and scales are asserted
to be finite first."""
import numpy as np
import torch

from tests.q8_reference import KIND, check_rows, f64

NAN_BYTE = 0x7f  # e4m3's NaN; 127 in int8


def check_finite_rows(q, scale, v, quant, rel, what):
    assert np.isfinite(v).all(), f"{what}: the reference itself is not finite"
    g, s = f64(q), f64(scale)
    assert np.isfinite(g).all(), f"{what}: {(~np.isfinite(g)).sum()} codes are NaN"
    assert np.isfinite(s).all(), f"{what}: {(~np.isfinite(s)).sum()} scales are not finite"
    check_rows(q, scale, v, quant, rel, what)


def nan_filled(rows, columns, quant, device="cuda"):
    """An 8-bit tensor of NaN bytes (int8: of 127s) and NaN scales, so that what
    a kernel leaves unwritten is seen."""
    q = torch.full((rows, columns), NAN_BYTE, dtype=torch.uint8, device=device)
    return q.view(KIND[quant]), torch.full((rows,), float("nan"), device=device)
