"""The product on 4-bit weights against the same sums in 64 bits."""
import numpy as np
import pytest
import torch

from tests import w4_reference as ref
from reduce_residual_rmsnorm_tw_gb300 import tw

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
X = {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8,
     "e4m3": torch.float8_e4m3fn}


def make(n, k, group, kind, seed=0):
    """(W4Weight, the weights in 64 bits)."""
    g = torch.Generator().manual_seed(seed + n + k)
    levels = torch.from_numpy(ref.LEVELS[kind]).float()
    v = levels[torch.randint(0, 8, (n, k), generator=g)]
    v = torch.where(torch.rand(n, k, generator=g) < 0.5, -v, v)
    if kind == "int4":
        v[torch.rand(n, k, generator=g) < 0.01] = -8
    s = (torch.rand(n, -(-k // group), generator=g) + 0.5).to(torch.bfloat16).float()
    w4 = tw.W4Weight.from_values(v.cuda(), s.cuda(), group, kind)
    return w4, ref.weights(v.double().numpy(), s.double().numpy(), group)


def make_x(t, k, xtype, seed=0):
    """(x, x_scale or None, x in 64 bits with its scales)."""
    g = torch.Generator().manual_seed(seed + 31 * t + k)
    v = torch.randn(t, k, generator=g)
    if xtype in ("bf16", "f32"):
        x, scale = v.to(X[xtype]), None
    else:
        x = (v * 40).round().clamp(-128, 127).to(X[xtype]) if xtype == "int8" else v.to(X[xtype])
        scale = torch.rand(t, generator=g) + 0.5
    x64 = x.float().double().numpy()
    if scale is not None:
        x64 = x64 * scale.double().numpy()[:, None]
    return x.cuda(), None if scale is None else scale.cuda(), x64


def check(out, x64, w64, group, fp32_x, what=""):
    got = out.float().double().cpu().numpy()
    want = x64 @ w64.T
    bound = ref.product_bound(x64, w64, want, group, out.dtype, fp32_x)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} off, worst {np.max(np.abs(got - want) / bound)}"


def run(t, n, k, group, kind, xtype, dtype, **kwargs):
    w4, w64 = make(n, k, group, kind)
    x, scale, x64 = make_x(t, k, xtype)
    out = torch.full((t, n), 9.0, dtype=DTYPES[dtype], device="cuda")
    tw.tw_gemm_w4(x, w4, out, x_scale=scale, **kwargs)
    check(out, x64, w64, group, xtype == "f32", (t, n, k, group, kind, xtype, dtype))


@pytest.mark.parametrize("kind", ["int4", "e2m1"])
@pytest.mark.parametrize("xtype", list(X))
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("t,n,k", [(1, 64, 128), (2, 100, 1040), (5, 1000, 528), (9, 33, 4096),
                                   (16, 4090, 272), (17, 48, 2064), (40, 130, 1600)])
def test_sizes_and_types(t, n, k, group, xtype, kind):
    run(t, n, k, group, kind, xtype, "f32" if (t + group) % 3 else "bf16")


@pytest.mark.parametrize("t,n,k", [(1, 1, 16), (3, 15, 48), (1, 8192, 1024), (1, 4096, 8192),
                                   (8, 1030, 8192), (11, 16, 65536), (1, 20000, 144),
                                   (33, 513, 8192), (300, 200, 400)])
@pytest.mark.parametrize("xtype", ["bf16", "f32", "int8"])
def test_shapes(t, n, k, xtype):
    run(t, n, k, 128, "int4", xtype, "bf16")


@pytest.mark.parametrize("max_sms", [1, 3, 76, 152])
@pytest.mark.parametrize("t,n,k", [(1, 1000, 2048), (20, 300, 1600)])
def test_budgets(t, n, k, max_sms):
    run(t, n, k, 64, "e2m1", "bf16", "f32", max_sms=max_sms)


@pytest.mark.parametrize("xtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_sms,k", [(1, 16384), (2, 32768), (3, 65536), (1, 65536)])
def test_long_rows_on_few_sms(max_sms, k, xtype):
    run(2, 150, k, 32, "int4", xtype, "f32", max_sms=max_sms)


def test_rows_outside_the_range_are_left_alone():
    w4, w64 = make(70, 256, 32, "int4")
    x, _, x64 = make_x(13, 256, "f32")
    out = torch.full((13, 70), 5.0, device="cuda")
    tw.tw_gemm_w4(x, w4, out, t0=4, t1=9)
    check(out[4:9], x64[4:9], w64, 32, True)
    assert torch.all(out[:4] == 5) and torch.all(out[9:] == 5)
    tw.tw_gemm_w4(x, w4, out, t0=3, t1=3)
    tw.tw_gemm_w4(x[:0], w4, out[:0])
    assert torch.all(out[:4] == 5)


def test_infinities_and_nans_stay_in_their_token_and_channel():
    w4, w64 = make(40, 300 // 16 * 16, 32, "int4")
    k = w4.k
    v, s, _ = ref.unpack(w4)
    s[7, 3] = np.nan
    w4 = tw.W4Weight.from_values(torch.from_numpy(v).float().cuda(),
                                 torch.from_numpy(s).float().cuda(), 32, "int4")
    w64 = ref.weights(v, s, 32)
    for dtype in DTYPES.values():
        x = torch.randn(6, k, generator=torch.Generator().manual_seed(2)).to(dtype)
        x[1, 5] = float("nan")
        x[2, 9] = float("inf")
        x[4, 100] = torch.finfo(dtype).max
        out = torch.empty(6, 40, device="cuda")
        tw.tw_gemm_w4(x.cuda(), w4, out)
        with np.errstate(invalid="ignore"):
            want = x.double().numpy() @ w64.T
        got = out.double().cpu().numpy()
        inside = np.abs(want) < 3.4e38
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(np.isinf(got), ~np.isnan(want) & ~inside)
        assert np.isfinite(got[[0, 3, 5]][:, np.arange(40) != 7]).all()


def test_nan_of_8_bits_and_scales_stay_in_their_token():
    w4, w64 = make(40, 208, 64, "e2m1")
    x, scale, x64 = make_x(9, 208, "e4m3")
    x[3, 100] = float("nan")
    scale[5], scale[6] = float("nan"), 0.0
    x64[6] = 0
    out = torch.empty(9, 40, device="cuda")
    tw.tw_gemm_w4(x, w4, out, x_scale=scale)
    assert out[[3, 5]].isnan().all() and not out[6].any()
    rest = [0, 1, 2, 4, 7, 8]
    check(out[rest], x64[rest], w64, 64, False)


@pytest.mark.parametrize("xtype", ["bf16", "f32"])
def test_small_x_keeps_its_bits(xtype):
    """Down to the magnitude that the header names, next to a large scale."""
    least = 2.0 ** (-110 if xtype == "bf16" else -96)
    v = torch.zeros(16, 64)
    v[:, 5] = 1
    w4 = tw.W4Weight.from_values(v.cuda(), torch.full((16, 2), 2.0 ** 90).cuda(), 32, "int4")
    x = torch.zeros(3, 64, dtype=X[xtype])
    x[:, 5] = torch.tensor([1.0, 1.9921875, 1.2421875 if xtype == "bf16" else 1 + 2.0 ** -23]) * least
    out = torch.empty(3, 16, device="cuda")
    tw.tw_gemm_w4(x.cuda(), w4, out)
    assert torch.equal(out.cpu(), (x[:, 5:6].double() * 2.0 ** 90).float().expand(3, 16))


def test_fp32_x_keeps_all_its_bits():
    """x of 24 significant bits against weights that pick one of them: exact."""
    k = 128
    v = torch.zeros(16, k)
    v[torch.arange(16), torch.arange(16) * 8 + 3] = 4.0
    w4 = tw.W4Weight.from_values(v.cuda(), torch.full((16, 4), 0.25).cuda(), 32, "int4")
    g = torch.Generator().manual_seed(4)
    bits = torch.randint(0x00800000, 0x7f800000, (50, k), generator=g, dtype=torch.int32)
    x = bits.view(torch.float32) * torch.sign(torch.randn(50, k, generator=g))
    x = torch.where(x.abs() < 2.0 ** -96, torch.ones_like(x), x)
    x = torch.where(x.abs() > 2.0 ** 125, torch.ones_like(x), x)
    out = torch.empty(50, 16, device="cuda")
    tw.tw_gemm_w4(x.cuda(), w4, out)
    assert torch.equal(out.cpu(), x[:, 3::8])


def test_one_large_value_beside_a_zero_weight():
    """A large x on a weight of 0 leaves no trace in the sum (exact products)."""
    w = torch.ones(32, 256)
    w[:, 17] = 0
    for kind in ("int4", "e2m1"):
        w4 = tw.W4Weight.from_values(w.cuda(), torch.ones(32, 8).cuda(), 32, kind)
        x = torch.ones(1, 256)
        x[0, 17] = 2.0 ** 30
        out = torch.empty(1, 32, device="cuda")
        tw.tw_gemm_w4(x.to(torch.bfloat16).cuda(), w4, out)
        assert torch.all(out == 255)


@pytest.mark.parametrize("t", [1, 7, 20])
def test_equal_calls_give_equal_bits_and_streams_do_not_matter(t):
    w4, w64 = make(3000, 2048, 128, "int4")
    x, _, x64 = make_x(t, 2048, "bf16")
    outs = [torch.empty(t, 3000, device="cuda") for _ in range(6)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, out in enumerate(outs):
        tw.tw_gemm_w4(x, w4, out, stream=streams[i % 2])
    torch.cuda.synchronize()
    check(outs[0], x64, w64, 128, False)
    for out in outs[1:]:
        assert torch.equal(out, outs[0])


@pytest.mark.parametrize("t", [1, 12])
def test_captured_and_replayed_on_new_inputs(t):
    w4, w64 = make(500, 1024, 64, "e2m1")
    x, scale, _ = make_x(t, 1024, "int8")
    out = torch.zeros(t, 500, device="cuda")
    tw.tw_gemm_w4(x, w4, out, x_scale=scale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tw.tw_gemm_w4(x, w4, out, x_scale=scale)
        tw.tw_gemm_w4(x, w4, out, x_scale=scale)
    x2, scale2, x64 = make_x(t, 1024, "int8", seed=77)
    x.copy_(x2)
    scale.copy_(scale2)
    graph.replay()
    torch.cuda.synchronize()
    check(out, x64, w64, 64, False)


def test_output_past_2_31_elements_and_packed_weights_past_2_31_bytes():
    n, k = 70000, 65536  # 2.4e9 bytes
    w4 = tw.W4Weight(n, k, 128, "int4")
    w4.packed.zero_()  # codes -8 with scale 0
    small, w64 = make(16, k, 128, "int4")
    w4.packed[-small.packed.numel():] = small.packed
    x, _, x64 = make_x(2, k, "bf16")
    out = torch.empty(2, n, device="cuda")
    tw.tw_gemm_w4(x, w4, out)
    check(out[:, -16:], x64, w64, 128, False)
    assert not out[:, :-16].any()
    w4, w64 = make(65536, 16, 32, "int4")
    x, _, x64 = make_x(33000, 16, "bf16")
    out = torch.empty(33000, 65536, dtype=torch.bfloat16, device="cuda")
    tw.tw_gemm_w4(x, w4, out)
    check(out[-3:], x64[-3:], w64, 32, False)
    check(out[:3], x64[:3], w64, 32, False)
