"""The 8-bit matrix product against the same product in 64 bits."""
import numpy as np
import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import tw
from tests.parity import SENTINEL
from tests.q8_reference import check_product, draw_8_bit, f64

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def run(T, N, K, quant, dtype, t0=0, t1=None, max_sms=None, seed=5):
    t1 = T if t1 is None else t1
    x, xs = draw_8_bit(T, K, quant, seed)
    w, ws = draw_8_bit(N, K, quant, seed + 1)
    out = torch.full((T, N), SENTINEL, dtype=DT[dtype], device="cuda")
    tw.tw_gemm_q8(x, xs, w, ws, out, t0, t1, max_sms=max_sms)
    torch.cuda.synchronize()
    check_product(out[t0:t1], x[t0:t1], xs[t0:t1], w, ws, f"{T}x{N}x{K} {quant} {dtype}")
    assert bool((torch.cat([out[:t0], out[t1:]]).float() == SENTINEL).all())
    assert tw.tw_device_status() == 0
    return out


# One token to several tiles of tokens; channels below, at and off a tile's
# edge, down to one; the shortest inner size, sizes off every slice, long ones.
SHAPES = [(1, 128, 128), (1, 1, 16), (2, 7, 48), (3, 8192, 1024), (8, 1000, 8192),
          (9, 130, 272), (16, 256, 144), (17, 129, 4096), (31, 64, 16), (33, 515, 1040),
          (64, 1024, 8192), (65, 127, 128), (100, 257, 2064), (128, 128, 128),
          (129, 300, 528), (192, 384, 256), (193, 255, 1008), (250, 999, 16), (256, 256, 384),
          (257, 513, 640), (333, 4090, 5120), (700, 96, 32), (1024, 1024, 1024)]


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_product_matches_reference(T, N, K, quant):
    run(T, N, K, quant, "f32" if (T + N) % 2 else "bf16")


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("max_sms", [1, 2, 5, 151, None])
def test_ranges_and_budgets(max_sms, quant):
    for T, t0, t1 in ((300, 7, 290), (5, 2, 3), (600, 0, 513)):
        run(T, 520, 1040, quant, "f32", t0, t1, max_sms=max_sms)


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
def test_repeated_calls_give_the_same_bits(quant):
    for T, N, K in ((4, 1024, 4096), (40, 2048, 4096), (400, 2048, 4096)):
        assert torch.equal(run(T, N, K, quant, "f32"), run(T, N, K, quant, "f32"))


def test_int8_is_exact_below_2_to_24():
    # Whole sums: with unit scales the fp32 output is the integer itself.
    T, N, K = 70, 300, 1024
    x, _ = draw_8_bit(T, K, "int8", 9)
    w, _ = draw_8_bit(N, K, "int8", 10)
    x[0], w[0] = -128, -128  # the largest sum: 2^24
    out = torch.empty(T, N, device="cuda")
    one = torch.ones(T, device="cuda"), torch.ones(N, device="cuda")
    tw.tw_gemm_q8(x, one[0], w, one[1], out)
    assert np.array_equal(f64(out), f64(x) @ f64(w).T)


@pytest.mark.parametrize("T", [3, 40, 300])
def test_nan_stays_in_its_row_and_column(T):
    # A NaN scale (a row that had none) and an e4m3 NaN value reach exactly
    # their row or column.
    N, K = 200, 256
    x, xs = draw_8_bit(T, K, "e4m3", 11)
    w, ws = draw_8_bit(N, K, "e4m3", 12)
    xs[1] = float("nan")
    w.view(torch.uint8)[150, 3] = 0x7f
    out = torch.empty(T, N, device="cuda")
    tw.tw_gemm_q8(x, xs, w, ws, out)
    bad = torch.isnan(out)
    want = torch.zeros_like(bad)
    want[1], want[:, 150] = True, True
    assert torch.equal(bad, want)


def test_captured_and_replayed_on_new_inputs():
    # A captured call reads the buffers' contents at replay, beside an eager
    # call on the same operands from another stream.
    T, N, K = 150, 260, 512
    x, xs = draw_8_bit(T, K, "int8", 13)
    w, ws = draw_8_bit(N, K, "int8", 14)
    out, out2 = (torch.empty(T, N, device="cuda") for _ in range(2))
    tw.tw_gemm_q8(x, xs, w, ws, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tw.tw_gemm_q8(x, xs, w, ws, out)
    x2, xs2 = draw_8_bit(T, K, "int8", 15)
    x.copy_(x2)
    xs.copy_(xs2)
    out.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g.replay()
    tw.tw_gemm_q8(x, xs, w, ws, out2, stream=side)
    torch.cuda.synchronize()
    check_product(out, x, xs, w, ws, "replayed")
    assert torch.equal(out, out2)


def test_empty_batch():
    x, xs = draw_8_bit(4, 64, "int8", 1)
    tw.tw_gemm_q8(x[:0], xs[:0], x, xs, torch.empty(0, 4, device="cuda"))
