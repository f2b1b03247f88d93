"""Every kernel is loaded when the library is set up, before any of them can be waiting
for another (a kernel that is loaded at its first launch may wait for running ones):
libtw.so on a stand-in for the CUDA runtime that notes what set-up asks for and what the
calls launch, in a child process."""
import os
import subprocess
import sys

import pytest

from reduce_residual_rmsnorm_tw_gb300 import build as twbuild

CHILD = """
import ctypes, sys
from ctypes import c_float, c_int, c_int64, c_void_p
lib = ctypes.CDLL(sys.argv[1])
BASE, MB = 0x7f0000000000, 1 << 28
at = lambda i: c_void_p(BASE + i * MB)
array = lambda *i: (c_void_p * len(i))(*[BASE + k * MB for k in i])
def step(T, H, dtype, q8, post, sms):
    name = "tw_fused_reduce_" + ("postnorm_" if post else "") + "add_rmsnorm" + ("_q8" if q8 else "")
    head = [array(0, 8), c_int(2)] + ([at(16), None, c_int64(1)] if post else [])
    head += [at(17), at(25), array(26)] + ([array(34)] if q8 else []) + [c_int(1), at(35)]
    size = [c_int64(T), c_int64(H)] + [c_float(v) for v in ((1e-5, 1e-5, 1., 1.) if post else (1e-5,))]
    tail = [c_int64(0), c_int64(T), c_int(sms), None, c_int(dtype)] + ([c_int(0)] if q8 else [])
    assert getattr(lib, name)(*head, *size, *tail) == 0
def gemm(T, N, K, group, xtype, wtype, sms):
    assert lib.tw_gemm_w4(at(0), at(1) if xtype > 1 else None, at(2), at(6), c_int64(T), c_int64(N),
                          c_int64(K), c_int(group), c_int64(0), c_int64(T), c_int(sms), None,
                          c_int(xtype), c_int(0), c_int(wtype)) == 0
def rows(name, dtype, wtype, group):
    assert getattr(lib, name)(at(0), at(4), c_int64(300), c_int64(1024), c_int(group),
                              c_int(1 << 30), None, c_int(dtype), c_int(wtype)) == 0
ALL = 1 << 30
for post in (False, True):
    for dtype in (0, 1):
        for q8 in (False, True):
            for H in (8, 256, 260, 504, 512, 1000, 1024, 2048, 2496, 2560, 4096, 5000, 6144, 8192,
                      12288, 16384):
                if H * (2, 4)[dtype] > 32768 or H * (2, 4)[dtype] % 16: continue
                for T in (1, 7, 100, 310, 620, 1300, 2600, 4100):
                    for sms in (1, 3, 8, 76, ALL):
                        step(T, H, dtype, q8, post, sms)
for wtype in (0, 1):
    for group in (32, 64, 128):
        for dtype in (0, 1):
            rows("tw_quantize_w4", dtype, wtype, group)
            rows("tw_dequantize_w4", dtype, wtype, group)
        for xtype in range(4):
            for T in (1, 9, 17, 25, 40):
                for sms in (1, 8, ALL): gemm(T, 500, 2048, group, xtype, wtype, sms)
"""


@pytest.fixture(scope="module")
def noted(tmp_path_factory):
    """(kernels that set-up asked for, kernels launched) by their mangled names."""
    fake = tmp_path_factory.mktemp("fake") / "liblog_cudart.so"
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "log_cudart.c")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", str(fake), src], check=True)
    env = dict(os.environ, LD_PRELOAD=str(fake), FAKE_FAIL="")
    out = subprocess.run([sys.executable, "-c", CHILD, twbuild.build()], env=env, check=True,
                         text=True, capture_output=True, timeout=300).stdout
    loaded, launched = set(), set()
    for line in out.splitlines():
        what, _, name = line.partition(" ")
        if what == "load":
            loaded.add(name)
        elif what == "launch":
            launched.add(name)
    return loaded, launched


def test_the_calls_reach_every_kind_of_kernel(noted):
    launched = noted[1]
    for kind in ("rows_kernel", "cluster_kernel", "15postnorm_kernel", "postnorm_rows_kernel",
                 "18quantize_w4_kernel", "dequantize_w4_kernel", "w4_gemm_kernel"):
        assert any(kind in name for name in launched), kind
    # The forms of the short rows' kernel for many rows (its last argument), each type.
    many = [n for n in launched if "15postnorm_kernel" in n and "Lb1EEEv" in n]
    assert len(many) == 24


def test_what_is_launched_was_loaded_at_set_up(noted):
    loaded, launched = noted
    assert launched <= loaded, sorted(launched - loaded)
