"""An operator whose kernels cannot be set up on a device refuses its calls, and
every other entry point still runs: libtw.so on a stand-in for the CUDA runtime
(tests/fake_cudart.c), in a child process."""
import os
import subprocess
import sys

import pytest

from reduce_residual_rmsnorm_tw_gb300 import build as twbuild

OK, UNSUP = 0, -5

CHILD = """
import ctypes, sys
from ctypes import c_float, c_int, c_int64, c_void_p
lib = ctypes.CDLL(sys.argv[1])
lib.tw_last_error_string.restype = ctypes.c_char_p
BASE, MB = 0x7f0000000000, 1 << 20
at = lambda i: c_void_p(BASE + i * MB)
array = lambda *i: (c_void_p * len(i))(*[BASE + k * MB for k in i])
def norm(T, q8):
    H, tail = 1024, (c_int64(0), c_int64(T), c_int(1 << 30), None, c_int(0))
    size = (c_int64(T), c_int64(H), c_float(1e-5))
    if q8:
        return lib.tw_fused_reduce_add_rmsnorm_q8(
            array(0, 16), c_int(2), at(32), at(48), array(64), array(80), c_int(1), at(96), *size,
            *tail, c_int(0))
    return lib.tw_fused_reduce_add_rmsnorm(
        array(0, 16), c_int(2), at(32), at(48), array(64), c_int(1), at(96), *size, *tail)
def rows():
    return lib.tw_quantize_rows_q8(at(0), at(16), at(32), c_int64(64), c_int64(1024), c_int64(0),
                                   c_int64(64), c_int(1 << 30), None, c_int(0), c_int(0))
def gemm(T):
    return lib.tw_gemm_q8(at(0), at(16), at(32), at(48), at(64), c_int64(T), c_int64(512),
                          c_int64(1024), c_int64(0), c_int64(T), c_int(1 << 30), None, c_int(0),
                          c_int(0))
for name, call in (("plain cluster", lambda: norm(4, False)), ("plain rows", lambda: norm(2000, False)),
                   ("norm cluster", lambda: norm(4, True)), ("norm rows", lambda: norm(2000, True)),
                   ("rows", rows), ("gemv", lambda: gemm(4)), ("gemm", lambda: gemm(40))):
    print("call", name, flush=True)
    print("status", call(), lib.tw_last_error_string().decode(), flush=True)
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    out = tmp_path_factory.mktemp("fake") / "libfake_cudart.so"
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "fake_cudart.c")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", str(out), src], check=True)
    return str(out)


def calls(fake, fail):
    """{call: (status, message, kernels launched)} with the set-up of kernels whose
    mangled name (or a driver entry point whose name) holds `fail` failing."""
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
    assert len(result) == 7
    return result


KERNEL = {"plain cluster": "cluster_kernel", "plain rows": "rows", "norm cluster": "cluster_kernel",
          "norm rows": "rows", "rows": "quantize_kernel", "gemv": "gemv_kernel",
          "gemm": "gemm_kernel"}


@pytest.mark.parametrize("fail,refused", [
    ("", []),
    ("gemm_kernel", ["gemm"]),
    ("cuTensorMapEncodeTiled", ["gemm"]),
    ("gemv_kernel", ["gemv"]),
    ("quantize_kernel", ["rows"]),
    # The rows kernel with 8-bit outputs (the template's last argument).
    ("rows_kernelI13__nv_bfloat16Li1ELi1ELi0ELb1E", ["norm cluster", "norm rows"]),
])
def test_one_operator_fails_alone(fake, fail, refused):
    for name, (status, message, launched) in calls(fake, fail).items():
        if name in refused:
            assert status == UNSUP and "unavailable" in message and launched == [], name
        else:
            assert status == OK, (name, message)
            assert len(launched) == 1 and KERNEL[name] in launched[0], (name, launched)


def test_cluster_kernel_with_8_bit_outputs_fails_alone(fake):
    # As without them: the rows kernel takes its calls.
    got = calls(fake, "cluster_kernelI13__nv_bfloat16Li1ELi2ELb1E")
    assert all(status == OK for status, _, _ in got.values())
    assert "cluster_kernel" in got["plain cluster"][2][0]
    assert "rows" in got["norm cluster"][2][0]
