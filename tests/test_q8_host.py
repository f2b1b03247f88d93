"""Refusals of the 8-bit entry points: every rule is checked on the host
before any CUDA call, so fake (never dereferenced) addresses suffice."""
import ctypes

import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import build as twbuild
from reduce_residual_rmsnorm_tw_gb300 import tw

OK, INVALID, ALIGN, ALIAS, UNSUP = 0, -1, -2, -3, -5
BASE, MB = 0x7f0000000000, 1 << 20


@pytest.fixture(scope="module")
def lib():
    twbuild.build()
    return tw.load()


def norm(lib, n_parts=2, n_out=1, T=4, H=64, eps=1e-6, t0=0, t1=None, max_sms=8, dtype=0,
         qtype=0, out=None, scale=None, residual_out=None):
    p_arr = (ctypes.c_void_p * 2)(BASE, BASE + MB)
    out = out or [BASE + (32 + k) * MB for k in range(n_out)]
    scale = [BASE + (40 + k) * MB for k in range(n_out)] if scale is None else scale
    o_arr = (ctypes.c_void_p * len(out))(*out)
    s_arr = (ctypes.c_void_p * len(scale))(*scale) if scale else None
    return lib.tw_fused_reduce_add_rmsnorm_q8(
        p_arr, n_parts, BASE + 64 * MB, BASE + 65 * MB, o_arr, s_arr, n_out,
        BASE + 66 * MB if residual_out is None else residual_out, T, H, eps, t0,
        T if t1 is None else t1, max_sms, None, dtype, qtype)


@pytest.mark.parametrize("kwargs,status", [
    ({"qtype": 2}, INVALID),
    ({"qtype": -1}, INVALID),
    ({"dtype": 2}, INVALID),
    ({"scale": []}, INVALID),                               # no scale array
    ({"scale": [0]}, INVALID),                              # a NULL scale
    ({"scale": [BASE + 40 * MB + 2]}, ALIGN),
    ({"scale": [BASE + 32 * MB + 240]}, ALIAS),             # inside out (4 x 64 bytes)
    ({"scale": [BASE + 66 * MB]}, ALIAS),                   # on residual_out
    ({"scale": [BASE + 64 * MB + 4]}, ALIAS),               # on the residual
    ({"n_out": 2, "scale": [BASE + 40 * MB, BASE + 40 * MB + 12]}, ALIAS),
    ({"n_out": 2, "out": [BASE + 32 * MB, BASE + 32 * MB + 240]}, ALIAS),
    ({"out": [BASE + 32 * MB + 8]}, ALIGN),
    ({"n_out": 9}, INVALID),
    ({"H": 12}, ALIGN),
    ({"H": 16392}, UNSUP),
    ({"t1": 5}, INVALID),
    ({"max_sms": 0}, INVALID),
    ({"eps": -1.0}, INVALID),
])
def test_norm_refusals(lib, kwargs, status):
    assert norm(lib, **kwargs) == status
    assert tw.tw_last_error_string() != ""


def test_norm_accepts_what_the_rules_allow(lib):
    # Empty ranges: no launch.  8-bit destinations are a byte per value, so
    # two of them may lie 256 bytes apart; residual_out may be the residual.
    assert norm(lib, t0=2, t1=2) == OK
    assert norm(lib, n_out=2, out=[BASE + 32 * MB, BASE + 32 * MB + 256], t1=0) == OK
    assert norm(lib, residual_out=BASE + 64 * MB, t1=0) == OK


def rows(lib, x=BASE, out=BASE + MB, scale=BASE + 2 * MB, T=4, H=64, t0=0, t1=None, max_sms=8,
         dtype=0, qtype=0):
    return lib.tw_quantize_rows_q8(x, out, scale, T, H, t0, T if t1 is None else t1, max_sms,
                                   None, dtype, qtype)


@pytest.mark.parametrize("kwargs,status", [
    ({"x": 0}, INVALID), ({"out": 0}, INVALID), ({"scale": 0}, INVALID),
    ({"H": 0}, INVALID), ({"T": -1, "t1": 0}, INVALID), ({"T": 1 << 46}, INVALID),
    ({"t0": 3, "t1": 2}, INVALID), ({"t0": -1}, INVALID), ({"t1": 5}, INVALID),
    ({"dtype": 3}, INVALID), ({"qtype": 2}, INVALID), ({"max_sms": 0}, INVALID),
    ({"H": 12}, ALIGN), ({"H": 6, "dtype": 1}, ALIGN), ({"x": BASE + 8}, ALIGN),
    ({"out": BASE + MB + 8}, ALIGN), ({"scale": BASE + 2 * MB + 1}, ALIGN),
    ({"H": 16392}, UNSUP), ({"H": 8196, "dtype": 1}, UNSUP),
    ({"out": BASE + 496}, ALIAS), ({"scale": BASE + MB + 252}, ALIAS), ({"scale": BASE}, ALIAS),
])
def test_quantize_refusals(lib, kwargs, status):
    assert rows(lib, **kwargs) == status
    assert tw.tw_last_error_string() != ""


def test_quantize_empty_range(lib):
    assert rows(lib, t0=4, t1=4) == OK
    assert rows(lib, T=0) == OK


def gemm(lib, x=BASE, xs=BASE + MB, w=BASE + 2 * MB, ws=BASE + 3 * MB, out=BASE + 4 * MB, T=4,
         N=8, K=64, t0=0, t1=None, max_sms=8, dtype=0, qtype=0):
    return lib.tw_gemm_q8(x, xs, w, ws, out, T, N, K, t0, T if t1 is None else t1, max_sms, None,
                          dtype, qtype)


@pytest.mark.parametrize("kwargs,status", [
    ({"x": 0}, INVALID), ({"xs": 0}, INVALID), ({"w": 0}, INVALID), ({"ws": 0}, INVALID),
    ({"out": 0}, INVALID), ({"N": 0}, INVALID), ({"K": 0}, INVALID), ({"K": -16}, INVALID),
    ({"N": 1 << 31}, INVALID), ({"T": 1 << 31}, INVALID), ({"T": (1 << 31) - 511}, INVALID),
    ({"N": (1 << 31) - 511}, INVALID), ({"T": (1 << 31) - 512, "N": 1 << 20}, INVALID),
    ({"T": -1, "t1": 0}, INVALID), ({"t0": 2, "t1": 1}, INVALID), ({"t1": 5}, INVALID),
    ({"dtype": 2}, INVALID), ({"qtype": 2}, INVALID), ({"max_sms": 0}, INVALID),
    ({"K": 72}, ALIGN), ({"K": 65552}, UNSUP), ({"x": BASE + 8}, ALIGN),
    ({"w": BASE + 2 * MB + 4}, ALIGN), ({"out": BASE + 4 * MB + 2}, ALIGN),
    ({"xs": BASE + MB + 2}, ALIGN), ({"ws": BASE + 3 * MB + 3}, ALIGN),
    ({"out": BASE + 240}, ALIAS), ({"out": BASE + 2 * MB + 496}, ALIAS),
    ({"out": BASE + MB}, ALIAS), ({"out": BASE + 3 * MB + 16}, ALIAS),
])
def test_gemm_refusals(lib, kwargs, status):
    assert gemm(lib, **kwargs) == status
    assert tw.tw_last_error_string() != ""


def test_gemm_empty_range(lib):
    assert gemm(lib, t0=1, t1=1) == OK
    assert gemm(lib, T=0) == OK
    # Any channel count, rows of out then not being 16-byte aligned.
    assert gemm(lib, N=7, t1=0) == OK


def test_binding_refusals():
    bf, q = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.int8)
    s, w = torch.zeros(4), torch.zeros(64, dtype=torch.bfloat16)
    def run(*args, **kwargs):
        with pytest.raises(ValueError) as e:
            tw.tw_fused_reduce_add_rmsnorm_q8(*args, eps=1e-6, **kwargs)
        return str(e.value)
    ok = dict(partials=[bf], residual=bf, weight=w, out=[q], out_scale=[s], residual_out=bf)
    assert "CUDA device" in run(**ok)                     # well formed, on the CPU
    assert "float32" in run(**{**ok, "out_scale": [s.double()]})
    assert "scale tensor" in run(**{**ok, "out_scale": []})
    assert "not supported" in run(**{**ok, "out": [bf]})
    assert "contiguous" in run(**{**ok, "out": [q, q.to(torch.float8_e4m3fn)],
                                  "out_scale": [s, s]})
    assert "contiguous" in run(**{**ok, "out": [torch.zeros(64, 4, dtype=torch.int8).t()]})
    assert "weight" in run(**{**ok, "weight": w[:8]})
    for bad in (dict(x=bf[0]), dict(x=bf.half()), dict(out=bf), dict(out_scale=s[:2]),
                dict(out=q[:, :32]), dict()):
        with pytest.raises(ValueError):
            tw.tw_quantize_rows_q8(**{**dict(x=bf, out=q, out_scale=s), **bad})
    out = torch.zeros(4, 8, dtype=torch.bfloat16)
    wq, ws = torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)
    for bad in (dict(w=wq[:, :48]), dict(w=wq.to(torch.float8_e4m3fn)), dict(x_scale=ws),
                dict(out=out.half()), dict(out=out[:, :4]), dict(x=bf), dict(w=wq.t()), dict()):
        with pytest.raises(ValueError):
            tw.tw_gemm_q8(**{**dict(x=q, x_scale=s, w=wq, w_scale=ws, out=out), **bad})
