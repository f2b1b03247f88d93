"""Weights into 4 bits and back on the GPU, bit for bit against the definition in
64 bits."""
import numpy as np
import pytest
import torch

from tests import w4_reference as ref
from reduce_residual_rmsnorm_tw_gb300 import tw

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def check(w, group, kind, **kwargs):
    """Quantise w (CPU) on the GPU: codes, scales and what they stand for."""
    n, k = w.shape
    w4 = tw.W4Weight(n, k, group, kind)
    w4.packed.fill_(0xa5)
    tw.tw_quantize_w4(w.cuda(), w4, **kwargs)
    values, scales, rest = ref.unpack(w4)
    want, want_scales = ref.quantise(w.double().numpy(), group, kind)
    assert np.array_equal(scales, want_scales, equal_nan=True)
    assert np.array_equal(values, want), f"{(values != want).sum()} codes"
    assert np.all(rest == 0)
    for dtype in DTYPES.values():
        out = torch.full((n, k), 7.0, dtype=dtype, device="cuda")
        tw.tw_dequantize_w4(w4, out, **kwargs)
        # q * s has 12 bits: exact in fp32, rounded to bf16 once.
        exact = torch.from_numpy(ref.weights(want, want_scales, group)).float().to(dtype)
        assert torch.equal(out.cpu().nan_to_num(-9.0), exact.nan_to_num(-9.0))


@pytest.mark.parametrize("kind", ["int4", "e2m1"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k,group", [(1, 16, 32), (16, 128, 64), (37, 400, 32), (333, 1040, 128),
                                       (3, 65536, 128), (2000, 528, 64)])
def test_normal_values(n, k, group, dtype, kind):
    g = torch.Generator().manual_seed(n + k)
    check(torch.randn(n, k, generator=g).to(DTYPES[dtype]), group, kind)


@pytest.mark.parametrize("kind", ["int4", "e2m1"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("exponent", [-116, -60, 0, 60, 120])
def test_middles_and_their_neighbours(dtype, kind, exponent):
    """Values on the middle between two codes, an ulp below and above it, under
    scales of every mantissa."""
    group = 32
    levels = ref.LEVELS[kind]
    middles = (levels[:-1] + levels[1:]) / 2
    n = 256
    w = np.zeros((n, group))
    for i in range(n):
        s = np.ldexp(1 + (i % 128) / 128, exponent)
        # A largest value whose scale is s: s * top has 11 bits at most.
        w[i, 0] = s * levels[-1]
        w[i, 1:8] = s * middles
        w[i, 8:15] = -s * middles * (1 + 2.0 ** -23)
        w[i, 15:22] = s * middles * (1 - 2.0 ** -24)
        w[i, 22:29] = s * middles * (1 + 2.0 ** -7 * (1 if i % 2 else -1))
    w[:, 0] = np.where(np.arange(n) < 128, w[:, 0], w[:, 0] * (1 + 2.0 ** -10))
    check(torch.from_numpy(w).to(DTYPES[dtype]), group, kind)


@pytest.mark.parametrize("kind", ["int4", "e2m1"])
def test_scales_on_the_middle_of_two_bf16(kind):
    """fp32 groups whose largest magnitude / top is the middle of two bf16 values, or
    rounds to it in fp32."""
    top = ref.TOP[kind]
    g = np.random.default_rng(3)
    middle = (1 + (2 * g.integers(0, 128, 4096) + 1) / 256) * 2.0 ** g.integers(-30, 30, 4096)
    most = (middle * top).astype(np.float32)
    most = most.view(np.int32) + g.integers(-2, 3, 4096).astype(np.int32)
    w = np.zeros((4096, 32), dtype=np.float32)
    w[:, 5] = most.view(np.float32)
    w[:, 9] = -w[:, 5] / 3
    check(torch.from_numpy(w), 32, kind)


@pytest.mark.parametrize("kind", ["int4", "e2m1"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_tiny_infinite_and_nan_groups(dtype, kind):
    w = torch.randn(40, 256, generator=torch.Generator().manual_seed(1)).to(DTYPES[dtype])
    w[3] = 0
    w[4, :32] = 0
    w[5, 32:64] = 2.0 ** -118
    w[6, 32:64] = 2.0 ** -117
    w[7, 70] = float("inf")
    w[8, 100] = float("-inf")
    w[9, 0] = float("nan")
    w[10, 255] = torch.finfo(w.dtype).max / 2
    w[11, :32] = -0.0
    for group in (32, 64, 128):
        check(w, group, kind)


@pytest.mark.parametrize("max_sms", [1, 7, 152])
def test_budgets_give_the_same(max_sms):
    g = torch.Generator().manual_seed(9)
    check(torch.randn(130, 1424, generator=g), 64, "int4", max_sms=max_sms)


@pytest.mark.parametrize("kind", ["int4", "e2m1"])
def test_tensors_aligned_to_16_bytes_only(kind):
    n, k = 20, 400
    g = torch.Generator().manual_seed(11)
    flat = torch.randn(n * k + 4, generator=g).cuda()
    w = flat[4:].view(n, k)
    assert w.data_ptr() % 32 == 16
    w4, ref4 = tw.W4Weight(n, k, 64, kind), tw.W4Weight(n, k, 64, kind)
    tw.tw_quantize_w4(w, w4)
    tw.tw_quantize_w4(w.clone(), ref4)
    assert torch.equal(w4.packed, ref4.packed)
    out = torch.empty(n * k + 8, device="cuda")[4:-4].view(n, k)
    tw.tw_dequantize_w4(w4, out)
    want = torch.empty(n, k, device="cuda")
    tw.tw_dequantize_w4(w4, want)
    assert torch.equal(out, want)


def test_past_2_31_elements():
    n, k = 40000, 65536  # 2.6e9 weights
    w4 = tw.W4Weight(n, k, 128, "e2m1")
    w = torch.zeros(n, k, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(5)
    tail = torch.randn(17, k, generator=g).to(torch.bfloat16)
    w[-17:] = tail.cuda()
    tw.tw_quantize_w4(w, w4)
    out = torch.empty_like(w)
    del w
    tw.tw_dequantize_w4(w4, out)
    want, scales = ref.quantise(tail.double().numpy(), 128, "e2m1")
    exact = torch.from_numpy(ref.weights(want, scales, 128)).float().to(torch.bfloat16)
    assert torch.equal(out[-17:].cpu(), exact)
    assert not out[:-17].any()
