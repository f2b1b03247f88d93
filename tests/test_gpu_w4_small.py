"""The 4-bit product under small scales: which bits of a group's contribution count."""
import numpy as np
import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import tw
from tests import w4_reference as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24  # half a step of fp32
N, K, GROUP = 48, 128, 32


def make(kind, exponent, seed):
    """Weights whose scales are 2^exponent times 1 to 2 (bf16 numbers)."""
    g = torch.Generator().manual_seed(seed)
    levels = torch.from_numpy(ref.LEVELS[kind]).float()
    v = levels[torch.randint(0, 8, (N, K), generator=g)]
    v = torch.where(torch.rand(N, K, generator=g) < 0.5, -v, v)
    s = torch.ldexp(1 + torch.randint(0, 128, (N, K // GROUP), generator=g) / 128.0,
                    torch.tensor(exponent)).to(torch.bfloat16).float()
    w4 = tw.W4Weight.from_values(v.cuda(), s.cuda(), GROUP, kind)
    return w4, ref.weights(v.double().numpy(), s.double().numpy(), GROUP)


@pytest.mark.parametrize("kind", ["int4", "e2m1"])
@pytest.mark.parametrize("exponent", [-133, -130, -126, -120, -112, -100])
def test_int8_x_loses_nothing(exponent, kind):
    """Whole numbers times scales: every group's sum is a multiple of 2^-141 of what it is
    held as (2^-14 for int8 and int4 times 2^-133, a bf16 number's last bit: 2^-147), which
    fp32 holds below its normal range too.  So the error is that of fp32 sums: of four
    groups' products and additions at most, and the last scale's."""
    w4, w64 = make(kind, exponent, 1)
    g = torch.Generator().manual_seed(2)
    x = torch.randint(-128, 128, (7, K), generator=g, dtype=torch.int32).to(torch.int8)
    x[0] = 0
    x[0, 5], x[1, :32] = 1, 1
    scale = torch.tensor([1.0, 1.0, 0.5, 3.0, 2.0 ** 60, 2.0 ** 100, 1.0])
    out = torch.empty(7, N, device="cuda")
    tw.tw_gemm_w4(x.cuda(), w4, out, x_scale=scale.cuda())
    x64, s64 = x.double().numpy(), scale.double().numpy()[:, None]
    want = x64 @ w64.T
    size = np.abs(x64) @ np.abs(w64).T
    # (Below its normal range fp32 rounds the scaled result to a multiple of 2^-149.)
    bound = (4 * U * size + U * np.abs(want)) * s64 * (1 + U) + 2.0 ** -150
    assert np.all(np.abs(out.double().cpu().numpy() - want * s64) <= bound)
    # One product: every bit of it.
    assert np.array_equal(out[0].double().cpu().numpy(), want[0])


@pytest.mark.parametrize("kind,step", [("int4", 2.0 ** -143), ("e2m1", 2.0 ** -150)])
@pytest.mark.parametrize("xtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("exponent", [-133, -128, -124, -120, -110])
def test_other_x_counts_to_the_step_that_the_header_names(exponent, xtype, kind, step):
    """A group's contribution, off by half of fp32's least step as it is held (2^-150, times
    2^7 for int4) besides the roundings of fp32 sums: up to three terms of x, four groups."""
    w4, w64 = make(kind, exponent, 3)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(6, K, generator=g)
    x = x.to({"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}[xtype])
    x64 = x.float().double().numpy()
    scale = torch.ones(6) if xtype == "e4m3" else None
    out = torch.empty(6, N, device="cuda")
    tw.tw_gemm_w4(x.cuda(), w4, out, x_scale=None if scale is None else scale.cuda())
    want = x64 @ w64.T
    bound = ref.product_bound(x64, w64, want, GROUP, torch.float32, xtype == "f32")
    terms = 3 if xtype == "f32" else 1
    bound = bound + (terms * (K // GROUP)) * step + 2.0 ** -150
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound)
