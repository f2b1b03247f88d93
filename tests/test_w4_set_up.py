"""The operators on 4-bit weights and the step with two norms where their kernels cannot
be set up: those calls refuse, every other one runs (libtw.so on a stand-in for the
CUDA runtime, in a child process)."""
import os
import subprocess
import sys

import pytest

from reduce_residual_rmsnorm_tw_gb300 import build as twbuild
from tests.test_q8_set_up import fake  # noqa: F401

OK, UNSUP = 0, -5

CHILD = """
import ctypes, sys
from ctypes import c_float, c_int, c_int64, c_void_p
lib = ctypes.CDLL(sys.argv[1])
lib.tw_last_error_string.restype = ctypes.c_char_p
BASE, MB = 0x7f0000000000, 1 << 20
at = lambda i: c_void_p(BASE + i * MB)
array = lambda *i: (c_void_p * len(i))(*[BASE + k * MB for k in i])
ALL = c_int(1 << 30)
def plain(T, H=1024):
    return lib.tw_fused_reduce_add_rmsnorm(
        array(0, 16), c_int(2), at(32), at(48), array(64), c_int(1), at(96), c_int64(T),
        c_int64(H), c_float(1e-5), c_int64(0), c_int64(T), ALL, None, c_int(0))
def post(T, H, sms=ALL):
    f = [c_float(v) for v in (1e-5, 1e-5, 1.0, 1.0)]
    return lib.tw_fused_reduce_postnorm_add_rmsnorm(
        array(0, 160), c_int(2), at(320), None, c_int64(1), at(321), at(480), array(481), c_int(1),
        at(640), c_int64(T), c_int64(H), *f, c_int64(0), c_int64(T), sms, None, c_int(0))
def quant(name):
    return getattr(lib, name)(at(0), at(32), c_int64(512), c_int64(1024), c_int(64), ALL, None,
                              c_int(0), c_int(0))
def gemm(T, K=1024, sms=ALL, xtype=0):
    return lib.tw_gemm_w4(at(0), None, at(128), at(512), c_int64(T), c_int64(512), c_int64(K),
                          c_int(64), c_int64(0), c_int64(T), sms, None, c_int(xtype), c_int(0),
                          c_int(0))
for name, call in (("plain", lambda: plain(4)), ("post short", lambda: post(4, 1024)),
                   ("post cluster", lambda: post(4, 8192)), ("post ring", lambda: post(2000, 8192)),
                   ("post long ring", lambda: post(2000, 16384)),
                   ("quantise", lambda: quant("tw_quantize_w4")),
                   ("read back", lambda: quant("tw_dequantize_w4")), ("product", lambda: gemm(4)),
                   ("product 20", lambda: gemm(20)), ("product 200", lambda: gemm(200)),
                   ("product long", lambda: gemm(1, 65536, c_int(1), 1))):
    print("call", name, flush=True)
    print("status", call(), lib.tw_last_error_string().decode(), flush=True)
"""

KERNEL = {"plain": "cluster_kernel", "post short": "15postnorm_kernel",
          "post cluster": "15postnorm_kernel", "post ring": "postnorm_rows_kernel",
          "post long ring": "postnorm_rows_kernel", "quantise": "18quantize_w4_kernel",
          "read back": "dequantize_w4_kernel", "product": "w4_gemm_kernel",
          "product 20": "w4_gemm_kernel", "product 200": "w4_gemm_kernel",
          "product long": "w4_gemm_kernel"}
POST = ["post short", "post cluster", "post ring", "post long ring"]
PRODUCT = ["product", "product 20", "product 200", "product long"]


def calls(fake, fail):  # noqa: F811
    lib = twbuild.build()
    env = dict(os.environ, LD_PRELOAD=fake, FAKE_FAIL=fail)
    out = subprocess.run([sys.executable, "-c", CHILD, lib], env=env, check=True, text=True,
                         capture_output=True, timeout=120).stdout
    result, launched = {}, []
    for line in out.splitlines():
        what, _, rest = line.partition(" ")
        if what == "call":
            name, launched = rest, []
        elif what == "launch":
            launched.append(rest)
        elif what == "status":
            status, _, message = rest.partition(" ")
            result[name] = (int(status), message, launched)
    assert list(result) == list(KERNEL)
    return result


@pytest.mark.parametrize("fail,refused", [
    ("", []), ("15postnorm_kernel", POST), ("postnorm_rows_kernel", POST),
    ("18quantize_w4_kernel", ["quantise", "read back"]),
    ("dequantize_w4_kernel", ["quantise", "read back"]), ("w4_gemm_kernel", PRODUCT)])
def test_one_operator_fails_alone(fake, fail, refused):  # noqa: F811
    for name, (status, message, launched) in calls(fake, fail).items():
        if name in refused:
            assert status == UNSUP and "unavailable" in message and launched == [], name
        else:
            assert status == OK, (name, message)
            assert len(launched) == 1 and KERNEL[name] in launched[0], (name, launched)
