"""The 4-bit entry points without a GPU: their refusals (every rule is checked on the
host before any CUDA call, so fake addresses suffice), and the packed form."""
import ctypes

import numpy as np
import pytest
import torch

from tests import w4_reference as ref
from reduce_residual_rmsnorm_tw_gb300 import build as twbuild
from reduce_residual_rmsnorm_tw_gb300 import layer_step, tw

OK, INVALID, ALIGN, ALIAS, UNSUP = 0, -1, -2, -3, -5
BASE, MB = 0x7f0000000000, 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    twbuild.build()
    return tw.load()


SHAPES = [({"N": 0}, INVALID), ({"N": -1}, INVALID), ({"N": (1 << 31) - 511}, INVALID),
          ({"K": 0}, INVALID), ({"K": -16}, INVALID), ({"K": 72}, ALIGN), ({"K": 65552}, UNSUP),
          ({"group": 0}, INVALID), ({"group": 16}, INVALID), ({"group": 256}, INVALID),
          ({"group": -32}, INVALID)]


@pytest.mark.parametrize("kwargs,status", SHAPES)
def test_bytes_refusals(lib, kwargs, status):
    a = {**dict(N=8, K=64, group=64), **kwargs}
    size = ctypes.c_size_t(7)
    assert lib.tw_w4_bytes(a["N"], a["K"], a["group"], ctypes.byref(size)) == status
    assert size.value == 7 and tw.tw_last_error_string() != ""


@pytest.mark.parametrize("n,k,group,want", [
    (1, 16, 32, 1024 + 128), (16, 128, 128, 1024 + 32), (17, 144, 64, 4 * (1024 + 64)),
    (8192, 8192, 128, 512 * 64 * 1056), ((1 << 31) - 512, 65536, 32, (1 << 27) * 512 * 1152 -
                                         32 * 512 * 1152)])
def test_bytes(lib, n, k, group, want):
    size = ctypes.c_size_t()
    assert lib.tw_w4_bytes(n, k, group, ctypes.byref(size)) == OK and size.value == want
    assert lib.tw_w4_bytes(n, k, group, None) == INVALID


def rows(lib, name, w=BASE, packed=BASE + MB, N=8, K=64, group=64, max_sms=8, dtype=0, wtype=0):
    first, second = (w, packed) if name == "tw_quantize_w4" else (packed, w)
    return getattr(lib, name)(first, second, N, K, group, max_sms, None, dtype, wtype)


@pytest.mark.parametrize("name", ["tw_quantize_w4", "tw_dequantize_w4"])
@pytest.mark.parametrize("kwargs,status", SHAPES + [
    ({"w": 0}, INVALID), ({"packed": 0}, INVALID), ({"max_sms": 0}, INVALID),
    ({"dtype": 2}, INVALID), ({"dtype": -1}, INVALID), ({"wtype": 2}, INVALID),
    ({"w": BASE + 8}, ALIGN), ({"packed": BASE + MB + 4}, ALIGN),
    ({"packed": BASE + 8 * 64 * 2 - 16}, ALIAS), ({"w": BASE + MB + 1024 + 48}, ALIAS)])
def test_rows_refusals(lib, name, kwargs, status):
    assert rows(lib, name, **kwargs) == status
    assert tw.tw_last_error_string() != ""


def gemm(lib, x=BASE, xs=0, packed=BASE + MB, out=BASE + 2 * MB, T=4, N=8, K=64, group=64, t0=0,
         t1=None, max_sms=8, xtype=0, dtype=0, wtype=0):
    return lib.tw_gemm_w4(x, xs or None, packed, out, T, N, K, group, t0, T if t1 is None else t1,
                          max_sms, None, xtype, dtype, wtype)


@pytest.mark.parametrize("kwargs,status", SHAPES + [
    ({"x": 0}, INVALID), ({"packed": 0}, INVALID), ({"out": 0}, INVALID),
    ({"T": -1, "t1": 0}, INVALID), ({"T": (1 << 31) - 511}, INVALID), ({"t0": -1}, INVALID),
    ({"t0": 3, "t1": 2}, INVALID), ({"t1": 5}, INVALID), ({"max_sms": 0}, INVALID),
    ({"T": (1 << 31) - 512, "N": 1 << 20}, INVALID), ({"xtype": 4}, INVALID),
    ({"xtype": -1}, INVALID), ({"dtype": 2}, INVALID), ({"wtype": -1}, INVALID),
    ({"xtype": 2}, INVALID), ({"xtype": 3}, INVALID), ({"xs": BASE + 3 * MB}, INVALID),
    ({"xtype": 2, "xs": BASE + 3 * MB + 2}, ALIGN), ({"x": BASE + 8}, ALIGN),
    ({"packed": BASE + MB + 8}, ALIGN), ({"out": BASE + 2 * MB + 2}, ALIGN),
    ({"out": BASE + 4 * 64 * 2 - 16}, ALIAS), ({"out": BASE + MB + 1024}, ALIAS),
    ({"xtype": 2, "xs": BASE + 2 * MB + 60}, ALIAS)])
def test_gemm_refusals(lib, kwargs, status):
    assert gemm(lib, **kwargs) == status
    assert tw.tw_last_error_string() != ""


def test_gemm_empty_range(lib):
    assert gemm(lib, t0=2, t1=2) == OK
    assert gemm(lib, T=0) == OK
    assert gemm(lib, N=7, t1=0, xtype=2, xs=BASE + 3 * MB) == OK


def test_binding_refusals():
    for bad in (dict(n=0), dict(k=24), dict(group=48), dict(k=1 << 17)):
        with pytest.raises(tw.TwError):
            tw.W4Weight(**{**dict(n=8, k=64, group=32, device="cpu"), **bad})
    with pytest.raises(ValueError):
        tw.W4Weight(8, 64, 32, "int3", "cpu")
    w4 = tw.W4Weight(8, 64, 32, "int4", "cpu")
    bf = torch.zeros(8, 64, dtype=torch.bfloat16)
    for call in (tw.tw_quantize_w4, lambda w, q: tw.tw_dequantize_w4(q, w)):
        for w in (bf, bf.half(), bf[:, :32], bf[:4], torch.zeros(64, 8, dtype=bf.dtype).t()):
            with pytest.raises(ValueError):
                call(w, w4)
    x, out, s = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 8), torch.zeros(4)
    q = x.to(torch.int8)
    for bad in (dict(), dict(x=x[0]), dict(x=x[:, :32]), dict(x=x.half()), dict(x_scale=s),
                dict(x=q), dict(x=q, x_scale=s[:2]), dict(x=q, x_scale=s.double()),
                dict(out=out.half()), dict(out=out[:, :4]), dict(out=out[:2]),
                dict(x=torch.zeros(64, 4, dtype=x.dtype).t())):
        with pytest.raises(ValueError):
            tw.tw_gemm_w4(**{**dict(x=x, w=w4, out=out), **bad})


def random_values(g, n, k, kind):
    levels = torch.from_numpy(ref.LEVELS[kind]).float()
    v = levels[torch.randint(0, 8, (n, k), generator=g)]
    v = torch.where(torch.rand(n, k, generator=g) < 0.5, -v, v)
    if kind == "int4":
        v[0, 0] = -8
    return v


@pytest.mark.parametrize("kind", ["int4", "e2m1"])
@pytest.mark.parametrize("n,k,group", [(1, 16, 32), (16, 128, 128), (37, 400, 32), (37, 400, 64),
                                       (50, 272, 128)])
def test_from_values_is_the_packed_form(n, k, group, kind):
    g = torch.Generator().manual_seed(n * k + group)
    v = random_values(g, n, k, kind)
    s = torch.rand(n, -(-k // group), generator=g).to(torch.bfloat16).float()
    w4 = tw.W4Weight.from_values(v, s, group, kind)
    values, scales, rest = ref.unpack(w4)
    assert np.array_equal(values, v.numpy()) and np.array_equal(scales, s.numpy())
    assert np.all(rest == 0)


def test_from_values_refuses_what_does_not_fit():
    v, s = torch.ones(8, 64), torch.ones(8, 2)
    for values, scale, kind in ((v * 8, s, "int4"), (v * 0.5, s, "int4"), (v * 2.5, s, "e2m1"),
                                (v * 8, s, "e2m1"), (v * float("nan"), s, "e2m1"),
                                (v, s[:, :1], "int4"), (v, s + 2.0 ** -10, "int4")):
        with pytest.raises(ValueError):
            tw.W4Weight.from_values(values, scale, 32, kind)
    nan = tw.W4Weight.from_values(v, s * float("nan"), 32, "int4")
    assert np.isnan(ref.unpack(nan)[1]).all()


def test_reference_rounds_middles_to_even_codes():
    w = np.zeros((1, 32))
    w[0, :5] = [7, 0.5, 1.5, 2.5, -3.5]
    assert np.array_equal(ref.quantise(w, 32, "int4")[0][0, :5], [7, 0, 2, 2, -4])
    w[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5]
    assert np.array_equal(ref.quantise(w, 32, "e2m1")[0][0, :8], [6, 0, 1, 1, 2, 2, 4, -4])


def test_many_tokens_go_to_the_library():
    assert layer_step.w4_library_tokens(4096, 4096) == 33
    assert layer_step.w4_library_tokens(8192, 8192) == 65
