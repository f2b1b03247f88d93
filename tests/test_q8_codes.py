"""Codes of finite rows are finite: the check itself (CPU), and every 8-bit
output of the operators in buffers that held NaN before (GPU)."""
import numpy as np
import pytest
import torch

import oracle
from reduce_residual_rmsnorm_tw_gb300 import inputs, layer_step, tw
from reduce_residual_rmsnorm_tw_gb300.inputs import Workload
from tests.q8_codes import NAN_BYTE, check_finite_rows, nan_filled
from tests.q8_reference import U, draw_8_bit, row_error
from tests.test_gpu_q8_chain import Chain


@pytest.mark.parametrize("byte", [0x7f, 0xff])
def test_check_refuses_nan_codes(byte):
    v = torch.linspace(-3, 3, 64, dtype=torch.float64).reshape(2, 32).numpy()
    s = torch.from_numpy(np.abs(v).max(axis=1) / 448).float()
    q = (torch.from_numpy(v).float() / s[:, None]).to(torch.float8_e4m3fn)
    rel = np.full(2, 3 * U)
    check_finite_rows(q, s, v, "e4m3", rel, "as it should be")
    q.view(torch.uint8)[1, 5] = byte
    with pytest.raises(AssertionError, match="1 codes are NaN"):
        check_finite_rows(q, s, v, "e4m3", rel, "one NaN")


def test_check_refuses_nan_scales():
    v = np.ones((1, 8))
    q = torch.full((1, 8), 127, dtype=torch.int8)
    with pytest.raises(AssertionError, match="scales"):
        check_finite_rows(q, torch.tensor([float("nan")]), v, "int8", np.full(1, 3 * U), "scale")


def norm_reference(p64, r64, w64, eps):
    """(rows, error of the largest value relative to it): the sum's error, and
    100 half steps for the multiplies, the inverse rms and the factor."""
    ref, _ = oracle.reordered(p64, r64, w64, eps, n_out=1)
    x = sum(p64) + r64
    return ref[0], 2 * row_error([p * w64 for p in p64 + [r64]], x * w64) + 100 * U


# The cluster kernel; the rows kernel with units of 1, 2 and 4 tokens, claimed
# units, two pipelines; a row that leaves threads idle.
@pytest.mark.gpu
@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("parts,T,H,dtype,max_sms",
                         [(3, 7, 1000, "bf16", None), (8, 64, 8192, "bf16", None),
                          (4, 300, 8192, "bf16", None), (2, 2048, 4096, "bf16", None),
                          (2, 700, 512, "bf16", 9), (2, 10100, 512, "bf16", None),
                          (4, 301, 5120, "f32", None), (5, 140, 16384, "bf16", 8)])
def test_norm_codes(parts, T, H, dtype, max_sms, quant):
    wl = Workload(f"codes_{parts}_{T}_{H}_{dtype}", parts, T, H, dtype, 1e-5, 1, 81)
    d = inputs.make_inputs(wl, device="cuda")
    q, s = nan_filled(T, H, quant)
    tw.tw_fused_reduce_add_rmsnorm_q8(d["partials"], d["residual"], d["weight"], [q], [s],
                                      torch.empty_like(d["residual"]), wl.eps, max_sms=max_sms)
    torch.cuda.synchronize()
    ref, rel = norm_reference([inputs.to_f64(p) for p in d["partials"]],
                              inputs.to_f64(d["residual"]), inputs.to_f64(d["weight"]), wl.eps)
    check_finite_rows(q, s, ref, quant, rel, wl.name)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("T,H,dtype", [(1, 8192, "bf16"), (37, 1000, "bf16"), (300, 8, "bf16"),
                                       (77, 264, "bf16"), (2500, 2056, "bf16"),
                                       (3, 16384, "bf16"), (700, 4, "f32"), (513, 1236, "f32"),
                                       (31, 8192, "f32")])
def test_quantised_codes(T, H, dtype, quant):
    g = torch.Generator()
    g.manual_seed(T * H)
    x = torch.randn(T, H, generator=g).to(inputs.DTYPES[dtype])
    for max_sms in (None, 3):
        q, s = nan_filled(T, H, quant)
        tw.tw_quantize_rows_q8(x.cuda(), q, s, max_sms=max_sms)
        # One division for the scale, one for the quotient.
        check_finite_rows(q, s, inputs.to_f64(x), quant, np.full(T, 3 * U), f"rows {T} {H}")


@pytest.mark.gpu
@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("T", [1, 70, 500])
def test_chain_codes(T, quant):
    c = Chain(T, 1024, 2000, quant, 91)
    for t in c.q:
        t.view(torch.uint8).fill_(NAN_BYTE)
    for t in c.s + [c.mid, c.down_out, c.res1, c.res2]:
        t.fill_(float("nan"))
    c.run()
    torch.cuda.synchronize()
    for t in c.q + c.s + [c.mid, c.down_out, c.res1, c.res2]:
        assert bool(torch.isfinite(t.float()).all())
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("T,split", [(600, None), (70, 3), (70, 0), (70, 70)])
def test_layer_step_codes(T, split, quant):
    wl = Workload(f"step_codes_{T}", 4, T, 2048, "bf16", 1e-5, 1, 98, partial_std=0.5)
    d = inputs.make_inputs(wl, device="cuda")
    x, xs = draw_8_bit(T, 1536, quant, 99)
    w, ws = draw_8_bit(2048, 1536, quant, 100)
    ws *= 0.01
    q, s = nan_filled(T, 2048, quant)
    res_out = torch.full_like(d["residual"], float("nan"))
    gemm, fused = torch.cuda.Stream(), torch.cuda.Stream(priority=-1)
    for st in (gemm, fused):
        st.wait_stream(torch.cuda.current_stream())
    layer_step.two_chunk_layer_step_q8(x, xs, w, ws, d["partials"], d["residual"],
                                       d["weight"], [q], [s], res_out, wl.eps, 16, gemm, fused,
                                       t_split=split)
    torch.cuda.synchronize()
    ref, rel = norm_reference([inputs.to_f64(p) for p in d["partials"]],
                              inputs.to_f64(d["residual"]), inputs.to_f64(d["weight"]), wl.eps)
    check_finite_rows(q, s, ref, quant, rel, "step")
    assert bool(torch.isfinite(res_out.float()).all())
