"""fp32 weights into 4 bits where a quotient leaves fp32's comfortable range, bit for bit
against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from tests.test_gpu_w4_rows import check
from tests.w4_reference import LEVELS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["int4", "e2m1"])
@pytest.mark.parametrize("most,small", [
    (1e30, 1e-20), (1e8, 1e-38), (1e8, 2.0 ** -126), (16.0, 2.0 ** -149), (14.0, 2.0 ** -149),
    (100.0, 3 * 2.0 ** -149), (2.0 ** 125, 2.0 ** -25), (2.0 ** 125, 2.0 ** -149),
    (3e38, 1e-10), (1.0, 2.0 ** -149), (2.0 ** -117, 2.0 ** -149)])
def test_quotients_that_underflow(most, small, kind):
    """A weight beside one up to 2^275 times as large stands for 0 and changes nothing
    beside it: of either sign, in every place of a word, alone and beside each other."""
    group = 32
    w = np.zeros((2 * group + 2, group), dtype=np.float32)
    for place in range(group):
        for negative in range(2):
            row = w[2 * place + negative]
            row[place] = -small if negative else small
            row[(place + 9) % group] = most
    for negative in range(2):
        w[2 * group + negative] = -small if negative else small
        w[2 * group + negative, 17] = -most
    check(torch.from_numpy(w), group, kind)


@pytest.mark.parametrize("kind", ["int4", "e2m1"])
@pytest.mark.parametrize("exponent", list(range(98, 126)))
def test_middles_under_large_scales(exponent, kind):
    """Values on the middle between two codes and up to four ulps beside it, under scales of
    every mantissa up to the largest that fp32 weights can have."""
    group, levels = 32, LEVELS[kind]
    middles = ((levels[:-1] + levels[1:]) / 2).astype(np.float32)
    rows = []
    for i in range(128):
        scale = np.ldexp(1 + i / 128, exponent)
        if scale * levels[-1] > np.finfo(np.float32).max:
            continue
        middle = middles * np.float32(scale)  # exact: 4 bits times 8
        for away in (-4, -2, -1, 0, 1, 2, 4):
            row = np.zeros(group, dtype=np.float32)
            row[0] = scale * levels[-1]  # 8 bits times 3 at most
            row[1:8] = (middle.view(np.int32) + np.int32(away)).view(np.float32)
            row[8:15] = -row[1:8]
            rows.append(row)
    check(torch.from_numpy(np.stack(rows)), group, kind)
