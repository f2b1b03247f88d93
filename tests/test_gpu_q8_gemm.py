"""The 8-bit matrix product against the same product in 64 bits."""
import numpy as np
import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import tw
from tests.parity import SENTINEL
from tests.q8_reference import check_product, draw_8_bit, f64, product, product_bound

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


# One token to several tiles of tokens; few tiles over a long K (split over
# clusters, shares of 8 columns up), many tiles; channels below, at and off a tile's
# edge, down to one; the shortest inner size, sizes off every slice, long ones.
SHAPES = [(1, 128, 128), (1, 1, 16), (2, 7, 48), (3, 8192, 1024), (8, 1000, 8192),
          (9, 130, 272), (16, 256, 144), (17, 129, 4096), (31, 64, 16), (33, 515, 1040),
          (64, 1024, 8192), (65, 127, 128), (100, 257, 2064), (128, 128, 128),
          (129, 300, 528), (192, 384, 256), (193, 255, 1008), (250, 999, 16), (256, 256, 384),
          (257, 513, 640), (333, 4090, 5120), (700, 96, 32), (1024, 1024, 1024),
          (4, 37, 65536), (20, 40, 65536), (12, 256, 8192), (40, 200, 8192), (64, 128, 4096),
          (90, 640, 8192), (120, 2048, 2048), (128, 1032, 6160), (300, 700, 8192), (600, 130, 4112),
          (2000, 264, 512), (1500, 4104, 256)]


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


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
def test_small_scales_keep_their_bits(quant):
    # Scales whose product is below fp32's normal range, the result is not.
    for T in (3, 40, 200):
        x, _ = draw_8_bit(T, 512, quant, 21)
        w, _ = draw_8_bit(264, 512, quant, 22)
        xs, ws = torch.full((T,), 2e-21, device="cuda"), torch.full((264,), 3e-20, device="cuda")
        out = torch.empty(T, 264, device="cuda")
        tw.tw_gemm_q8(x, xs, w, ws, out)
        want, size = product(x, xs, w, ws)
        raw = np.abs(f64(x)) @ np.abs(f64(w)).T if quant == "int8" else np.full_like(want, np.inf)
        big = np.abs(want) > 1e-37  # fp32's normal range ends at 1.2e-38
        # Sums of sum|x w| <= 2^27 times 2e-21 times 3e-20 stay normal at every
        # step, so the bound of any product holds: e4m3's sum rounds relative
        # to sum|x w|, which may be far above |want| where terms cancel.
        err, bound = np.abs(f64(out) - want), product_bound(want, size, raw, 512, out.dtype)
        assert big.any() and np.all(err[big] <= bound[big])


def test_offsets_past_2_to_31():
    # 2.2e9 output elements; 2.6e9 bytes of x.  Sampled rows.
    for T, N, K, dtype in ((270000, 8192, 16, "bf16"), (40000, 24, 65536, "f32")):
        x = torch.randint(-128, 128, (T, K), dtype=torch.int8, device="cuda")
        w = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda")
        xs, ws = torch.rand(T, device="cuda"), torch.rand(N, device="cuda")
        out = torch.empty(T, N, dtype=DT[dtype], device="cuda")
        tw.tw_gemm_q8(x, xs, w, ws, out)
        rows = torch.tensor([0, 1, T // 2, T - 130, T - 2, T - 1], device="cuda")
        check_product(out[rows], x[rows], xs[rows], w, ws, f"{T}x{N}x{K}")
        del x, w, out


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


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
def test_two_streams_at_once_give_the_same_bits(quant):
    # Products of different cuts (lone CTAs, pairs, split K, few tokens) queued
    # on two streams without a pause, the GPU's caches holding neither's inputs.
    shapes = [(256, 2304, 4096), (128, 520, 8192), (6, 4096, 4096), (60, 300, 8192),
              (700, 1000, 2064)]
    ops, want, outs = [], [], []
    for i, (T, N, K) in enumerate(shapes):
        x, xs = draw_8_bit(T, K, quant, 50 + i)
        w, ws = draw_8_bit(N, K, quant, 70 + i)
        out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        tw.tw_gemm_q8(x, xs, w, ws, out)
        torch.cuda.synchronize()
        check_product(out, x, xs, w, ws, f"{T}x{N}x{K} {quant}")
        ops.append((x, xs, w, ws))
        want.append(out)
        outs.append([torch.empty_like(out) for _ in range(2)])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    flush = torch.empty(1 << 26, dtype=torch.int32, device="cuda")
    for _ in range(8):
        flush.fill_(1)
        for pair in outs:
            for o in pair:
                o.zero_()
        torch.cuda.synchronize()
        for i in range(len(shapes)):
            tw.tw_gemm_q8(*ops[i], outs[i][0], stream=streams[0])
            j = len(shapes) - 1 - i
            tw.tw_gemm_q8(*ops[j], outs[j][1], stream=streams[1])
        torch.cuda.synchronize()
        for w, pair in zip(want, outs):
            assert all(torch.equal(w, o) for o in pair)
    assert tw.tw_device_status() == 0


def test_empty_batch():
    x, xs = draw_8_bit(4, 64, "int8", 1)
    tw.tw_gemm_q8(x[:0], xs[:0], x, xs, torch.empty(0, 4, device="cuda"))
