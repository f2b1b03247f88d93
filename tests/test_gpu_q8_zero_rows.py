"""Rows at the edges of what a scale can hold: largest magnitudes one step to
either side of 2^-117, and norms whose 1 / rms makes of an ordinary row one that is
zero, infinite or NaN.  Scale and codes have to say the same as the plain step's
values: 0 and zeros, or NaN and zeros."""
import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import inputs, tw
from tests.q8_reference import KIND, TOP, f64

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -117
# One token and more than the cluster kernel takes, the latter also on few SMs
# (two pipelines per CTA).
LAUNCHES = [(3, None), (300, None), (300, 8)]


def norm(x, w, quant, eps, max_sms=None):
    """(codes, scales, the plain step's values) of rows x without a residual."""
    T, H = x.shape
    zero = torch.zeros_like(x)
    q = torch.full((T, H), 77, dtype=torch.uint8, device="cuda").view(KIND[quant])
    s = torch.full((T,), -3.0, device="cuda")
    tw.tw_fused_reduce_add_rmsnorm_q8([x], zero, w, [q], [s], torch.empty_like(x), eps,
                                      max_sms=max_sms)
    y = torch.empty_like(x)
    tw.tw_fused_reduce_add_rmsnorm([x], zero, w, [y], torch.empty_like(x), eps, max_sms=max_sms)
    return f64(q), f64(s), y.float().cpu()


def rows(T, largest, dtype):
    """T rows of 1024 values from -largest to largest, the last of them largest."""
    x = torch.linspace(-0.9, 0.9, 1024).expand(T, 1024) * torch.tensor(largest, dtype=torch.float32)
    x = x.to(inputs.DTYPES[dtype])
    x[:, 1000] = largest
    return x.cuda()


def below(dtype):
    """The value before 2^-117."""
    return TINY * (1 - torch.finfo(inputs.DTYPES[dtype]).eps / 2)


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantised_rows_about_the_limit(dtype, quant):
    for largest, live in ((TINY, True), (below(dtype), False),
                          (TINY * (1 + torch.finfo(inputs.DTYPES[dtype]).eps), True)):
        x = rows(5, largest, dtype)
        q = torch.full((5, 1024), 77, dtype=torch.uint8, device="cuda").view(KIND[quant])
        s = torch.full((5,), -3.0, device="cuda")
        tw.tw_quantize_rows_q8(x, q, s)
        if live:
            assert (f64(s) == f64(x[:, 1000].float() / TOP[quant])).all()
            assert (f64(q)[:, 1000] == TOP[quant]).all()
        else:
            assert (f64(s) == 0).all() and (f64(q) == 0).all()


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,max_sms", LAUNCHES)
def test_norm_of_rows_about_the_limit(T, max_sms, dtype, quant):
    # max |x w| is exactly 2^-117 (y: 316 times that), then one step below.
    w = torch.ones(1024, dtype=inputs.DTYPES[dtype], device="cuda")
    q, s, _ = norm(rows(T, TINY, dtype), w, quant, 1e-5, max_sms)
    want = TINY / 1e-5 ** 0.5 / TOP[quant]
    assert (abs(s - want) <= 1e-6 * want).all() and (q[:, 1000] == TOP[quant]).all()
    q, s, _ = norm(rows(T, below(dtype), dtype), w, quant, 1e-5, max_sms)
    assert (s == 0).all() and (q == 0).all()


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,max_sms", LAUNCHES)
def test_norm_whose_values_are_tiny(T, max_sms, dtype, quant):
    # Rows of +-2^50 have rms 2^50, so y is the weight, with signs: a scale from
    # 2^-116 / top up, none for 2^-118, although x * weight is large.
    sign = torch.where(torch.arange(1024) % 2 == 0, 1.0, -1.0).expand(T, 1024)
    x = (sign * 2.0 ** 50).to(inputs.DTYPES[dtype]).cuda()
    for power, live in ((-116, True), (-118, False), (-126, False)):
        w = torch.full((1024,), 2.0 ** power, dtype=x.dtype, device="cuda")
        q, s, _ = norm(x, w, quant, 1e-5, max_sms)
        if live:
            want = 2.0 ** power / TOP[quant]
            assert (abs(s - want) <= 1e-6 * want).all() and (abs(q) == TOP[quant]).all()
        else:
            assert (s == 0).all() and (q == 0).all()


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,max_sms", LAUNCHES)
def test_norm_whose_sum_of_squares_leaves_fp32(T, max_sms, dtype, quant):
    w = torch.ones(1024, dtype=inputs.DTYPES[dtype], device="cuda")
    # Above fp32: 1 / rms is 0, and so is every value.
    q, s, y = norm(rows(T, 2.0 ** 100, dtype), w, quant, 1e-5, max_sms)
    assert (y == 0).all() and (s == 0).all() and (q == 0).all()
    # Below it, without an eps: 1 / rms is infinite, and so are the values.
    q, s, y = norm(rows(T, 2.0 ** -90, dtype), w, quant, 0.0, max_sms)
    assert torch.isinf(y[:, 1000]).all()
    assert (s != s).all() and (q == 0).all()
    # A row of zeros without an eps: 0 times infinity.
    q, s, y = norm(rows(T, 0.0, dtype), w, quant, 0.0, max_sms)
    assert torch.isnan(y).all()
    assert (s != s).all() and (q == 0).all()
    # The same row with an eps.
    q, s, y = norm(rows(T, 0.0, dtype), w, quant, 1e-5, max_sms)
    assert (y == 0).all() and (s == 0).all() and (q == 0).all()
    # x * weight overflows: the row counts as one that holds an infinity.
    q, s, _ = norm(rows(T, 2.0 ** 60, dtype), w * 2.0 ** 70, quant, 1e-5, max_sms)
    assert (s != s).all() and (q == 0).all()
