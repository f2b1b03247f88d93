"""The sums of the 8-bit product where fp32 is short of bits: whole numbers up to
2^24 with odd low bits (exact), and terms of one sign over a long K (the stated
bound).  3 tokens take the dot-product or the few-token matrix path, 7 the latter,
40 a split of K, 300 pairs of CTAs."""
import numpy as np
import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import tw
from tests.q8_reference import f64

pytestmark = pytest.mark.gpu
TOKENS = [1, 3, 7, 8, 16, 40, 300]


def whole(rows, K, low, high, g):
    return torch.randint(low, high + 1, (rows, K), generator=g, dtype=torch.int32).to(torch.int8)


def run(x, w):
    """The fp32 product with unit scales, in 64 bits."""
    T, N = x.shape[0], w.shape[0]
    out = torch.empty(T, N, device="cuda")
    tw.tw_gemm_q8(x.cuda(), torch.ones(T, device="cuda"), w.cuda(), torch.ones(N, device="cuda"),
                  out)
    return f64(out)


@pytest.mark.parametrize("N", [40, 300, 2048])
@pytest.mark.parametrize("T", TOKENS)
def test_whole_sums_to_2_to_24_are_exact(T, N):
    # 1024 products of 115..127 squared: sums of 13.5 to 16.5 million, whose
    # last bits are the first that a shorter accumulator would lose.
    g = torch.Generator()
    g.manual_seed(T * N)
    x, w = whole(T, 1024, 115, 127, g), whole(N, 1024, 115, 127, g)
    want = f64(x) @ f64(w).T
    assert 2 ** 23 < want.min() and want.max() < 2 ** 24 and (want % 2 == 1).any()
    assert np.array_equal(run(x, w), want)


@pytest.mark.parametrize("T", TOKENS)
def test_sums_that_climb_and_cancel_are_exact(T):
    # Up to 12 to 16 million over the first 992 elements, then down again by products
    # of -128 and of either sign: what was lost at the top would show below.
    g = torch.Generator()
    g.manual_seed(T)
    N, K = 300, 1968
    x, w = whole(T, K, 113, 127, g), whole(N, K, 113, 127, g)
    x[:, 992:] = -x[:, 992:]
    w[:, 1900:] = whole(N, 68, -128, 127, g)
    want = f64(x) @ f64(w).T
    partial = np.cumsum(f64(x)[:, None, :] * f64(w)[None, :20, :], axis=2)
    assert np.abs(partial).max() < 2 ** 24 and np.abs(want).max() < 2 ** 22
    assert np.array_equal(run(x, w), want)


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("K", [1024, 8192, 65536])
@pytest.mark.parametrize("T", TOKENS)
def test_terms_of_one_sign_keep_the_stated_bound(T, K, quant):
    # Each running sum rounds or truncates by up to 2^-23 of itself at each of
    # its K / 16 steps (and the joins, fewer than 32); terms of one sign keep it as
    # large as it can be.  Unit scales, fp32 out: the last rounding is in the 32.
    g = torch.Generator()
    g.manual_seed(K + T)
    N = 136
    if quant == "int8":
        x, w = whole(T, K, 1, 127, g), whole(N, K, 1, 127, g)
    else:
        x, w = (torch.rand(n, K, generator=g).mul(440).add(1).to(torch.float8_e4m3fn)
                for n in (T, N))
    want = f64(x) @ f64(w).T
    err = np.abs(run(x, w) - want)
    worst = (err / want).max() * 2 ** 24
    print(f"{quant} T {T} K {K}: off by {worst:.2f} x 2^-24 of the sum")
    assert (err <= (K / 16 + 32) * 2.0 ** -23 * want).all()
