"""Row quantisation's codes against the exact quotient v * top / max|v|: bf16 rows,
many of whose values lie in the very middle of two codes, get the definition's code
everywhere; fp32 rows the code of the quotient rounded to fp32."""
import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import inputs, tw
from tests.q8_reference import KIND, TOP

pytestmark = pytest.mark.gpu


def round_8_bit(q, quant):
    """fp64 quotients to the nearest 8-bit value, ties to even, as bytes with one
    zero (every e4m3 magnitude below 2^-6 is a multiple of 2^-9)."""
    if quant == "int8":
        return q.round().to(torch.int8).view(torch.uint8)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    codes = ((q / step).round() * step).clamp(-448, 448).float()
    return one_zero(codes.to(KIND[quant]).view(torch.uint8), quant)  # exact


def one_zero(b, quant):
    return torch.where((b & 0x7f) == 0, torch.zeros_like(b), b) if quant == "e4m3" else b


def check(x, quant, max_sms=None):
    T, H = x.shape
    q = torch.full((T, H), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((T,), -3.0, device="cuda")
    tw.tw_quantize_rows_q8(x.cuda(), q.view(KIND[quant]), s, max_sms=max_sms)
    got, m = one_zero(q.cpu(), quant), x.float().abs().amax(1)
    assert torch.equal(s.cpu(), m / TOP[quant])  # IEEE division
    # Whole numbers of at most 33 and 29 bits decide on which side of a middle
    # v * top / m lies, so 53 bits of it do.
    exact = x.double() * TOP[quant] / m.double()[:, None]
    if x.dtype == torch.bfloat16:
        bad = got != round_8_bit(exact, quant)
    else:
        # Before it is rounded to fp32 the quotient may be off by 2^-44, in rows
        # above 2^100 (whose top / max has fewer bits) by 2^-28.
        off = torch.where(m > 2.0 ** 100, 2.0 ** -28, 2.0 ** -44).double()[:, None]
        either = [round_8_bit((exact * (1 + d)).float().double(), quant) for d in (-off, off)]
        bad = (got != either[0]) & (got != either[1])
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} codes are off"


def from_bits(bits, dtype):
    if dtype == torch.bfloat16:
        return bits.to(torch.int16).view(dtype)
    return bits.to(torch.int32).view(dtype)


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("exponent", [-117, -100, -61, -60, 0, 59, 60, 61, 100, 127])
def test_every_bf16_mantissa_by_every_bf16_mantissa(exponent, quant):
    # Row i: the maximum 2^exponent * (1 + i / 128), then every mantissa in the
    # binades below it that bf16 has (at most 20: 448 / 2^20 is below half of
    # e4m3's least step), with both signs in turn.
    binades = min(20, exponent + 126)
    top = ((exponent + 127) << 7) | torch.arange(128)
    below = (exponent + 127 - 1 - torch.arange(binades))[:, None] * 128 + torch.arange(128)
    below = below.flatten() | (torch.arange(128 * binades) % 2) << 15
    rows = torch.cat([top[:, None].expand(128, 8), below.expand(128, -1)], 1)
    check(from_bits(rows, torch.bfloat16), quant)


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("exponent", [-116, -61, 0, 59, 60, 127])
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
    rows = torch.minimum(torch.cat([m[:, None], rows], 1), m[:, None])
    check(torch.nn.functional.pad(rows, (0, -rows.shape[1] % 4)), quant)


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
