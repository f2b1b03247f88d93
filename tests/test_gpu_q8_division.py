"""Row quantisation against fp32 division, bit for bit: scale = max|v| / top and
code = v / scale rounded to nearest even, values that lie in the very middle of
two codes among them (bf16 rows hold many)."""
import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import inputs, tw
from tests.q8_reference import KIND, TOP

pytestmark = pytest.mark.gpu


def by_division(x, quant):
    """(codes as bytes, scales) of the rows of x, on the CPU (IEEE division)."""
    v = x.float()
    s = v.abs().amax(1) / TOP[quant]
    q = v / s[:, None]
    q = q.round().to(torch.int8) if quant == "int8" else q.clamp(-448, 448).to(KIND[quant])
    return q.view(torch.uint8), s


def check(x, quant, max_sms=None):
    T, H = x.shape
    q = torch.full((T, H), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((T,), -3.0, device="cuda")
    tw.tw_quantize_rows_q8(x.cuda(), q.view(KIND[quant]), s, max_sms=max_sms)
    want_q, want_s = by_division(x, quant)
    got = q.cpu()
    if quant == "e4m3":  # zeros of either sign
        got, want_q = (torch.where((b & 0x7f) == 0, torch.zeros_like(b), b) for b in (got, want_q))
    assert torch.equal(s.cpu(), want_s)
    bad = got != want_q
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} codes are not the division's"


def from_bits(bits, dtype):
    if dtype == torch.bfloat16:
        return bits.to(torch.int16).view(dtype)
    return bits.to(torch.int32).view(dtype)


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("exponent", [-100, -61, -60, -59, 0, 100, 127])
def test_every_bf16_mantissa_by_every_bf16_mantissa(exponent, quant):
    # Row i: the maximum 2^exponent * (1 + i / 128), then every mantissa in
    # the 20 binades below it (448 / 2^20 is below half of e4m3's least step),
    # with both signs in turn.
    top = ((exponent + 127) << 7) | torch.arange(128)
    below = (exponent + 127 - 1 - torch.arange(20))[:, None] * 128 + torch.arange(128)
    below = below.flatten() | (torch.arange(2560) % 2) << 15
    rows = torch.cat([top[:, None].expand(128, 8), below.expand(128, 2560)], 1)
    check(from_bits(rows, torch.bfloat16), quant)


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("exponent", [-116, -61, -59, 0, 127])
def test_fp32_values_about_every_middle(exponent, quant):
    # The fp32 values nearest to the middle of every two codes and up to four
    # steps to either side, under row maxima of any mantissa.
    g = torch.Generator()
    g.manual_seed(exponent + 200)
    T = 200
    mantissa = torch.randint(0, 1 << 23, (T,), generator=g)
    mantissa[:2] = torch.tensor([0, (1 << 23) - 1])
    m = from_bits(((exponent + 127) << 23) | mantissa, torch.float32)
    if quant == "int8":
        middle = torch.arange(127) + 0.5
    else:
        codes = torch.arange(0x7f, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        middle = (codes[1:] + codes[:-1]) / 2
    near = (middle.double() * (m.double() / TOP[quant])[:, None]).float().view(torch.int32)
    steps = torch.arange(-4, 5, dtype=torch.int32)
    rows = (near[:, :, None] + steps).flatten(1).clamp(min=0).view(torch.float32)
    rows = torch.cat([m[:, None], rows], 1)
    rows = torch.minimum(rows, m[:, None])
    rows = torch.nn.functional.pad(rows, (0, -rows.shape[1] % 4))
    check(rows, quant)


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(300, 8), (77, 264), (37, 1000), (150, 2056), (40, 4096),
                                 (1024, 8192)])
def test_normal_rows(T, H, dtype, quant):
    g = torch.Generator()
    g.manual_seed(T + H)
    x = torch.randn(T, H, generator=g).to(inputs.DTYPES[dtype])
    for max_sms in (None, 3):
        check(x, quant, max_sms)


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
def test_longest_rows(quant):
    g = torch.Generator()
    g.manual_seed(7)
    check(torch.randn(20, 16384, generator=g).bfloat16(), quant)
    check(torch.randn(20, 8192, generator=g), quant)
