"""Refusals of the step with two norms: every rule is checked on the host before any
CUDA call, so fake (never dereferenced) addresses suffice."""
import ctypes

import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import build as twbuild
from reduce_residual_rmsnorm_tw_gb300 import tw

OK, INVALID, ALIGN, ALIAS, UNSUP = 0, -1, -2, -3, -5
BASE, MB = 0x7f0000000000, 1 << 20
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    twbuild.build()
    return tw.load()


def call(lib, q8=False, n_parts=2, post=BASE + 70 * MB, gate=BASE + 80 * MB, gate_tokens=1, n_out=1,
         T=4, H=64, post_eps=1e-6, eps=1e-6, block_scale=1.0, residual_scale=1.0, t0=0, t1=None,
         max_sms=8, dtype=0, qtype=0, out=None, scale=None, residual_out=BASE + 66 * MB):
    p_arr = (ctypes.c_void_p * 2)(BASE, BASE + MB)
    out = out or [BASE + (32 + k) * MB for k in range(n_out)]
    o_arr = (ctypes.c_void_p * len(out))(*out)
    head = [p_arr, n_parts, post or None, gate or None, gate_tokens, BASE + 64 * MB,
            BASE + 65 * MB, o_arr]
    tail = [n_out, residual_out, T, H, post_eps, eps, block_scale, residual_scale, t0,
            T if t1 is None else t1, max_sms, None, dtype]
    if not q8:
        return lib.tw_fused_reduce_postnorm_add_rmsnorm(*head, *tail)
    scale = [BASE + (40 + k) * MB for k in range(n_out)] if scale is None else scale
    s_arr = (ctypes.c_void_p * len(scale))(*scale) if scale else None
    return lib.tw_fused_reduce_postnorm_add_rmsnorm_q8(*head, s_arr, *tail, qtype)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kwargs,status", [
    ({"n_parts": 0}, INVALID), ({"n_parts": 17}, INVALID), ({"n_out": 9}, INVALID),
    ({"dtype": 2}, INVALID), ({"T": -1, "t1": 0}, INVALID), ({"H": 0}, INVALID),
    ({"H": 16392}, UNSUP), ({"H": 12}, ALIGN), ({"t0": -1}, INVALID), ({"t1": 5}, INVALID),
    ({"t0": 3, "t1": 2}, INVALID), ({"max_sms": 0}, INVALID), ({"eps": -1.0}, INVALID),
    ({"eps": INF}, INVALID), ({"post_eps": -1e-9}, INVALID), ({"post_eps": NAN}, INVALID),
    ({"post_eps": INF, "post": 0}, INVALID), ({"block_scale": NAN}, INVALID),
    ({"block_scale": INF}, INVALID), ({"residual_scale": -INF}, INVALID),
    ({"residual_scale": NAN}, INVALID), ({"gate_tokens": 0}, INVALID),
    ({"gate_tokens": -3}, INVALID), ({"post": BASE + 70 * MB + 8}, ALIGN),
    ({"gate": BASE + 80 * MB + 4}, ALIGN), ({"residual_out": BASE + 66 * MB + 8}, ALIGN),
    ({"post": BASE + 66 * MB + 496}, ALIAS), ({"post": BASE + 32 * MB}, ALIAS),
    ({"gate": BASE + 66 * MB + 496}, ALIAS),
    # The last of four rows of the gate on the output.
    ({"gate": BASE + 66 * MB - 384}, ALIAS), ({"gate": BASE + 66 * MB - 128, "gate_tokens": 3}, ALIAS),
    ({"residual_out": BASE + 64 * MB + 16}, ALIAS), ({"residual_out": BASE}, ALIAS),
    ({"residual_out": BASE + 32 * MB}, ALIAS),
])
def test_refusals(lib, kwargs, status, q8):
    assert call(lib, q8, **kwargs) == status
    assert tw.tw_last_error_string() != ""


@pytest.mark.parametrize("kwargs,status", [
    ({"qtype": 2}, INVALID), ({"scale": []}, INVALID), ({"scale": [0]}, INVALID),
    ({"scale": [BASE + 40 * MB + 2]}, ALIGN), ({"scale": [BASE + 70 * MB + 64]}, ALIAS),
    ({"scale": [BASE + 80 * MB + 64]}, ALIAS), ({"scale": [BASE + 66 * MB]}, ALIAS)])
def test_refusals_8_bits(lib, kwargs, status):
    assert call(lib, True, **kwargs) == status


def test_accepts_what_the_rules_allow(lib):
    for q8 in (False, True):
        assert call(lib, q8, t0=2, t1=2) == OK
        assert call(lib, q8, T=0) == OK
        assert call(lib, q8, t1=0, gate=0, gate_tokens=0) == OK
        assert call(lib, q8, t1=0, post=0, gate=0) == OK
        assert call(lib, q8, t1=0, residual_out=BASE + 64 * MB) == OK
        # One row of the gate ends where the output begins; weight as post_weight.
        assert call(lib, q8, t1=0, gate=BASE + 66 * MB - 128, gate_tokens=4) == OK
        assert call(lib, q8, t1=0, post=BASE + 65 * MB) == OK
        assert call(lib, q8, t1=0, block_scale=0.0, residual_scale=-2.0) == OK


def test_binding_refusals():
    bf, w, s = (torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16),
                torch.zeros(4))
    q = torch.zeros(4, 64, dtype=torch.int8)
    ok = dict(partials=[bf], residual=bf, weight=w, out=[bf], residual_out=bf, eps=1e-6)
    bad = [dict(), dict(partials=[]), dict(out=[]), dict(residual=bf[0]),
           dict(residual=bf.half()), dict(post_weight=w[:8]), dict(post_weight=w.float()),
           dict(gate=bf[:3]), dict(gate=bf.float()), dict(gate=bf, gate_tokens=2),
           dict(gate=bf, gate_tokens=0), dict(gate=w), dict(weight=w[:8]),
           dict(out=[bf.float()]), dict(residual_out=bf[:, :32])]
    for b in bad:
        with pytest.raises(ValueError):
            tw.tw_fused_reduce_postnorm_add_rmsnorm(**{**ok, **b})
    ok = {**ok, "out": [q], "out_scale": [s]}
    for b in bad + [dict(out_scale=[]), dict(out_scale=[s.double()]), dict(out=[bf])]:
        with pytest.raises(ValueError):
            tw.tw_fused_reduce_postnorm_add_rmsnorm_q8(**{**ok, **b})
