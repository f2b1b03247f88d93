"""Thin ctypes binding of libtw.so (argument marshalling only).

Every function keeps the name of the C entry point it calls.  Tensors are
torch tensors used only as device memory: the binding reads their pointers,
shapes and dtypes, the library checks the rules of ``include/tw.h`` and runs
every step of the computation in its CUDA kernels.  There is no fallback: if
``libtw.so`` is missing the first call raises.
"""
import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtw.so")

TW_BF16, TW_F32 = 0, 1
PATHS = {"auto": 0, "rows": 1, "warp": 2, "cluster": 3}
MAX_PARTS, MAX_OUTS = 16, 8
STATUS_NAMES = {0: "TW_OK", -1: "TW_ERR_INVALID_ARG", -2: "TW_ERR_ALIGNMENT",
                -3: "TW_ERR_ALIAS", -4: "TW_ERR_CUDA", -5: "TW_ERR_UNSUPPORTED"}
_DTYPES = {torch.bfloat16: TW_BF16, torch.float32: TW_F32}
TW_INT8, TW_E4M3 = 0, 1
_QTYPES = {torch.int8: TW_INT8, torch.float8_e4m3fn: TW_E4M3}
WTYPES = {"int4": 0, "e2m1": 1}
_XTYPES = {torch.bfloat16: 0, torch.float32: 1, torch.int8: 2, torch.float8_e4m3fn: 3}
# The current stream's handle without a Stream object around it (a decode step's
# kernel is over in the time that takes).  The call is private to torch: where it
# is missing, the public one serves.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_ALL_SMS = 1 << 30  # clamped to the device's SM count by the library


class TwError(RuntimeError):
    """A libtw.so call returned a status other than TW_OK."""

    def __init__(self, status, message):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_lib = None


def load():
    """Load libtw.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build the CUDA library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    pp = ctypes.POINTER(ctypes.c_void_p)
    common = [pp, ctypes.c_int, vp, vp, pp, ctypes.c_int, vp, i64, i64,
              ctypes.c_float, i64, i64, ctypes.c_int, vp]
    for name, extra in (("tw_fused_reduce_add_rmsnorm_bf16", []),
                        ("tw_fused_reduce_add_rmsnorm_f32", []),
                        ("tw_fused_reduce_add_rmsnorm", [ctypes.c_int]),
                        ("tw_fused_reduce_add_rmsnorm_colsplit", [ctypes.c_int]),
                        ("tw_fused_reduce_add_rmsnorm_ex",
                         [ctypes.c_int, ctypes.c_int, vp])):
        fn = getattr(lib, name)
        fn.argtypes = common + extra
        fn.restype = ctypes.c_int
    lib.tw_fused_reduce_add_rmsnorm_flags.argtypes = common + [
        ctypes.c_int, vp, i64, ctypes.c_uint32]
    lib.tw_fused_reduce_add_rmsnorm_flags.restype = ctypes.c_int
    lib.tw_set_ready.argtypes = [vp, i64, i64, ctypes.c_uint32, vp]
    lib.tw_set_ready.restype = ctypes.c_int
    lib.tw_fused_reduce_add_rmsnorm_q8.argtypes = [
        pp, ctypes.c_int, vp, vp, pp, pp, ctypes.c_int, vp, i64, i64, ctypes.c_float, i64, i64,
        ctypes.c_int, vp, ctypes.c_int, ctypes.c_int]
    lib.tw_fused_reduce_add_rmsnorm_q8.restype = ctypes.c_int
    lib.tw_quantize_rows_q8.argtypes = [vp, vp, vp, i64, i64, i64, i64, ctypes.c_int, vp,
                                        ctypes.c_int, ctypes.c_int]
    lib.tw_quantize_rows_q8.restype = ctypes.c_int
    lib.tw_gemm_q8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, ctypes.c_int, vp,
                               ctypes.c_int, ctypes.c_int]
    lib.tw_gemm_q8.restype = ctypes.c_int
    floats = [ctypes.c_float] * 4
    lib.tw_fused_reduce_postnorm_add_rmsnorm.argtypes = [
        pp, ctypes.c_int, vp, vp, i64, vp, vp, pp, ctypes.c_int, vp, i64, i64, *floats, i64, i64,
        ctypes.c_int, vp, ctypes.c_int]
    lib.tw_fused_reduce_postnorm_add_rmsnorm.restype = ctypes.c_int
    lib.tw_fused_reduce_postnorm_add_rmsnorm_q8.argtypes = [
        pp, ctypes.c_int, vp, vp, i64, vp, vp, pp, pp, ctypes.c_int, vp, i64, i64, *floats, i64,
        i64, ctypes.c_int, vp, ctypes.c_int, ctypes.c_int]
    lib.tw_fused_reduce_postnorm_add_rmsnorm_q8.restype = ctypes.c_int
    lib.tw_w4_bytes.argtypes = [i64, i64, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]
    lib.tw_w4_bytes.restype = ctypes.c_int
    for name in ("tw_quantize_w4", "tw_dequantize_w4"):
        fn = getattr(lib, name)
        fn.argtypes = [vp, vp, i64, i64, ctypes.c_int, ctypes.c_int, vp, ctypes.c_int,
                       ctypes.c_int]
        fn.restype = ctypes.c_int
    lib.tw_gemm_w4.argtypes = [vp, vp, vp, vp, i64, i64, i64, ctypes.c_int, i64, i64,
                               ctypes.c_int, vp, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    lib.tw_gemm_w4.restype = ctypes.c_int
    lib.tw_split_launch.argtypes = [pp, ctypes.c_int, vp, vp, pp, ctypes.c_int,
                                    vp, i64, i64, ctypes.c_float, i64,
                                    ctypes.c_int, vp, vp, ctypes.c_int]
    lib.tw_split_launch.restype = ctypes.c_int
    lib.tw_fused_reduce_add_rmsnorm_host.argtypes = [
        pp, ctypes.c_int, vp, vp, pp, ctypes.c_int, vp, i64, i64, ctypes.c_float,
        i64, i64, ctypes.c_int, vp, ctypes.c_size_t, i64, vp, ctypes.c_int]
    lib.tw_fused_reduce_add_rmsnorm_host.restype = ctypes.c_int
    lib.tw_fused_reduce_add_rmsnorm_host_noalloc.argtypes = [
        pp, ctypes.c_int, vp, vp, pp, ctypes.c_int, vp, i64, i64, ctypes.c_float,
        i64, i64, ctypes.c_int, i64, vp, ctypes.c_int]
    lib.tw_fused_reduce_add_rmsnorm_host_noalloc.restype = ctypes.c_int
    lib.tw_host_workspace_bytes.argtypes = [ctypes.c_int, ctypes.c_int, i64, i64,
                                            ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]
    lib.tw_host_workspace_bytes.restype = ctypes.c_int
    lib.tw_device_status.argtypes = [ctypes.c_int]
    lib.tw_device_status.restype = ctypes.c_int
    lib.tw_last_error_string.argtypes = []
    lib.tw_last_error_string.restype = ctypes.c_char_p
    lib.tw_version.argtypes = []
    lib.tw_version.restype = ctypes.c_int
    _lib = lib
    return lib


def _check(rc):
    if rc != 0:
        raise TwError(rc, load().tw_last_error_string().decode())


def _stream_handle(stream):
    if stream is None:
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _marshal(partials, residual, weight, out, residual_out, on_device=True):
    """Pointer arrays and (T, H, dtype) from tensors; shapes must agree.  The
    device entry points take tensors on the current CUDA device; the host
    entry points (on_device=False) take pinned CPU tensors."""
    partials, out = list(partials), list(out)
    if not partials or not out:
        raise ValueError("need at least one partial and one destination")
    if residual.dim() != 2:
        raise ValueError("residual must be [T, H]")
    T, H = residual.shape
    dtype = residual.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"dtype {dtype} not supported (bfloat16 or float32)")
    for name, ts in (("partials", partials), ("out", out),
                     ("residual_out", [residual_out])):
        for t in ts:
            if t.shape != (T, H) or t.dtype != dtype or not t.is_contiguous():
                raise ValueError(f"{name}: every tensor must be a contiguous "
                                 f"[{T}, {H}] {dtype} tensor")
    if (weight.shape != (H,) or weight.dtype != dtype
            or not weight.is_contiguous()):
        raise ValueError(f"weight must be a contiguous [{H}] {dtype} tensor")
    every = partials + out + [residual, weight, residual_out]
    if on_device:
        if any(not t.is_cuda for t in every):
            raise ValueError("every tensor must be on the current CUDA device")
        dev = torch.cuda.current_device()
        if any(t.device.index != dev for t in every):
            raise ValueError(f"every tensor must be on the current CUDA device (cuda:{dev})")
    elif any(t.is_cuda or not t.is_pinned() for t in every):
        raise ValueError("every tensor must be a pinned (page-locked) CPU tensor")
    p_arr = (ctypes.c_void_p * len(partials))(*[t.data_ptr() for t in partials])
    o_arr = (ctypes.c_void_p * len(out))(*[t.data_ptr() for t in out])
    return p_arr, len(partials), o_arr, len(out), T, H, _DTYPES[dtype]


def tw_fused_reduce_add_rmsnorm_ex(partials, residual, weight, out,
                                   residual_out, eps, t0=0, t1=None,
                                   max_sms=None, stream=None, path="auto",
                                   smid_log=None):
    """Fused reduce + residual add + RMSNorm on rows [t0, t1), kernel chosen
    by ``path`` ("auto", "rows", "warp" or "cluster").  ``smid_log`` is an optional int32
    device tensor with at least max_sms entries."""
    p_arr, n, o_arr, n_out, T, H, dt = _marshal(partials, residual, weight,
                                                out, residual_out)
    rc = load().tw_fused_reduce_add_rmsnorm_ex(
        p_arr, n, residual.data_ptr(), weight.data_ptr(), o_arr, n_out,
        residual_out.data_ptr(), T, H, eps, t0, T if t1 is None else t1,
        _ALL_SMS if max_sms is None else max_sms, _stream_handle(stream), dt,
        PATHS[path], None if smid_log is None else smid_log.data_ptr())
    _check(rc)


def tw_fused_reduce_add_rmsnorm(partials, residual, weight, out, residual_out,
                                eps, t0=0, t1=None, max_sms=None, stream=None):
    """Fused reduce + residual add + RMSNorm on rows [t0, t1) (kernel chosen
    by the library)."""
    p_arr, n, o_arr, n_out, T, H, dt = _marshal(partials, residual, weight,
                                                out, residual_out)
    rc = load().tw_fused_reduce_add_rmsnorm(
        p_arr, n, residual.data_ptr(), weight.data_ptr(), o_arr, n_out,
        residual_out.data_ptr(), T, H, eps, t0, T if t1 is None else t1,
        _ALL_SMS if max_sms is None else max_sms, _stream_handle(stream), dt)
    _check(rc)


def tw_fused_reduce_add_rmsnorm_colsplit(partials, residual, weight, out,
                                         residual_out, eps, t0=0, t1=None,
                                         max_sms=None, stream=None):
    """The fused step for zero-padded column-split partials: partial r is
    nonzero only in columns [r*H//N, (r+1)*H//N), and only those are read."""
    p_arr, n, o_arr, n_out, T, H, dt = _marshal(partials, residual, weight,
                                                out, residual_out)
    rc = load().tw_fused_reduce_add_rmsnorm_colsplit(
        p_arr, n, residual.data_ptr(), weight.data_ptr(), o_arr, n_out,
        residual_out.data_ptr(), T, H, eps, t0, T if t1 is None else t1,
        _ALL_SMS if max_sms is None else max_sms, _stream_handle(stream), dt)
    _check(rc)


def tw_fused_reduce_add_rmsnorm_flags(partials, residual, weight, out,
                                      residual_out, eps, ready, block_tokens,
                                      epoch, t0=0, t1=None, max_sms=None,
                                      stream=None):
    """The fused step gated by readiness flags: token t is read only once
    ``ready[t // block_tokens]`` (an int32 CUDA tensor) has reached ``epoch``."""
    p_arr, n, o_arr, n_out, T, H, dt = _marshal(partials, residual, weight,
                                                out, residual_out)
    if ready.dtype != torch.int32 or not ready.is_cuda:
        raise ValueError("ready must be an int32 CUDA tensor")
    rc = load().tw_fused_reduce_add_rmsnorm_flags(
        p_arr, n, residual.data_ptr(), weight.data_ptr(), o_arr, n_out,
        residual_out.data_ptr(), T, H, eps, t0, T if t1 is None else t1,
        _ALL_SMS if max_sms is None else max_sms, _stream_handle(stream), dt,
        ready.data_ptr(), block_tokens, epoch & 0xFFFFFFFF)
    _check(rc)


def tw_set_ready(ready, epoch, first_block=0, n_blocks=None, stream=None):
    """Raise ``ready[first_block:first_block + n_blocks]`` (an int32 CUDA
    tensor) to ``epoch`` with release stores, after the work queued earlier
    on ``stream``: the producer side of tw_fused_reduce_add_rmsnorm_flags."""
    if ready.dtype != torch.int32 or not ready.is_cuda or not ready.is_contiguous():
        raise ValueError("ready must be a contiguous int32 CUDA tensor")
    if n_blocks is None:
        n_blocks = ready.numel() - first_block
    if first_block < 0 or n_blocks < 0 or first_block + n_blocks > ready.numel():
        raise ValueError("flag range outside the ready tensor")
    _check(load().tw_set_ready(ready.data_ptr(), first_block, n_blocks, epoch & 0xFFFFFFFF,
                               _stream_handle(stream)))


def _typed(name, dtype):
    def call(partials, residual, weight, out, residual_out, eps, t0=0, t1=None,
             max_sms=None, stream=None):
        if residual.dtype != dtype:
            raise ValueError(f"{name} takes {dtype} tensors")
        p_arr, n, o_arr, n_out, T, H, _ = _marshal(partials, residual, weight,
                                                   out, residual_out)
        rc = getattr(load(), name)(
            p_arr, n, residual.data_ptr(), weight.data_ptr(), o_arr, n_out,
            residual_out.data_ptr(), T, H, eps, t0, T if t1 is None else t1,
            _ALL_SMS if max_sms is None else max_sms, _stream_handle(stream))
        _check(rc)
    call.__name__ = name
    call.__doc__ = f"The fused step on {dtype} tensors (C entry point {name})."
    return call


tw_fused_reduce_add_rmsnorm_bf16 = _typed("tw_fused_reduce_add_rmsnorm_bf16",
                                          torch.bfloat16)
tw_fused_reduce_add_rmsnorm_f32 = _typed("tw_fused_reduce_add_rmsnorm_f32",
                                         torch.float32)


def _on_current_device(*tensors):
    dev = torch.cuda.current_device() if tensors[0].is_cuda else None
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError("every tensor must be on the current CUDA device")


def _quantised(q, name="out"):
    """The tw_qtype of an 8-bit tensor."""
    qt = _QTYPES.get(q.dtype)
    if qt is None:
        raise ValueError(f"{name}: dtype {q.dtype} not supported (int8 or float8_e4m3fn)")
    return qt


def _dense(name, t, shape, dtype):
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} {dtype} tensor")


@functools.cache
def _pointer_array(n):
    return ctypes.c_void_p * n


def _pointers(name, tensors, shape, dtype, dev):
    """The pointers of alike tensors on device ``dev`` as a ctypes array."""
    ptrs = _pointer_array(len(tensors))()
    for i, t in enumerate(tensors):
        if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {list(shape)} {dtype} tensors")
        if t.get_device() != dev:
            raise ValueError("every tensor must be on the current CUDA device")
        ptrs[i] = t.data_ptr()
    return ptrs


def tw_fused_reduce_add_rmsnorm_q8(partials, residual, weight, out, out_scale,
                                   residual_out, eps, t0=0, t1=None,
                                   max_sms=None, stream=None):
    """The fused step with 8-bit outputs: every tensor of ``out`` ([T, H], all
    int8 or all float8_e4m3fn) and its ``out_scale`` ([T] float32) hold the
    normalised rows as values times one scale per token."""
    if residual.dim() != 2:
        raise ValueError("residual must be [T, H]")
    shape, dtype = residual.shape, residual.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"dtype {dtype} not supported (bfloat16 or float32)")
    T, H = shape
    n, n_out = len(partials), len(out)
    if not n or not n_out or len(out_scale) != n_out:
        raise ValueError("need at least one partial, one destination and a scale tensor for "
                         "each destination")
    qt = _quantised(out[0])
    # The device every tensor has to be on (-1: the tensors are on the CPU,
    # which _on_current_device refuses once their shapes are checked).
    dev = torch.cuda.current_device() if residual.is_cuda else -1
    p_arr = _pointers("partials", partials, shape, dtype, dev)
    o_arr = _pointers("out", out, shape, out[0].dtype, dev)
    s_arr = _pointers("out_scale", out_scale, (T,), torch.float32, dev)
    _dense("residual", residual, shape, dtype)
    _dense("residual_out", residual_out, shape, dtype)
    _dense("weight", weight, (H,), dtype)
    _on_current_device(residual, weight, residual_out)
    if T == 0:
        return
    _check(load().tw_fused_reduce_add_rmsnorm_q8(
        p_arr, n, residual.data_ptr(), weight.data_ptr(), o_arr, s_arr, n_out,
        residual_out.data_ptr(), T, H, eps, t0, T if t1 is None else t1,
        _ALL_SMS if max_sms is None else max_sms, _stream_handle(stream), _DTYPES[dtype], qt))


def tw_quantize_rows_q8(x, out, out_scale, t0=0, t1=None, max_sms=None, stream=None):
    """Rows [t0, t1) of ``x`` ([T, H] bfloat16 or float32) quantised into
    ``out`` ([T, H] int8 or float8_e4m3fn) and ``out_scale`` ([T] float32)."""
    if x.dim() != 2 or x.dtype not in _DTYPES:
        raise ValueError("x must be a [T, H] bfloat16 or float32 tensor")
    T, H = x.shape
    _dense("x", x, x.shape, x.dtype)
    qt = _quantised(out)
    _dense("out", out, x.shape, out.dtype)
    _dense("out_scale", out_scale, (T,), torch.float32)
    _on_current_device(x, out, out_scale)
    if T == 0:
        return
    _check(load().tw_quantize_rows_q8(
        x.data_ptr(), out.data_ptr(), out_scale.data_ptr(), T, H, t0, T if t1 is None else t1,
        _ALL_SMS if max_sms is None else max_sms, _stream_handle(stream), _DTYPES[x.dtype], qt))


def tw_gemm_q8(x, x_scale, w, w_scale, out, t0=0, t1=None, max_sms=None, stream=None):
    """out[t, n] = x_scale[t] * w_scale[n] * sum_k x[t, k] * w[n, k] on rows
    [t0, t1): ``x`` [T, K] and ``w`` [N, K] both int8 or both float8_e4m3fn,
    the scales float32, ``out`` [T, N] bfloat16 or float32."""
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x must be [T, K] and w [N, K]")
    T, K = x.shape
    N = w.shape[0]
    qt = _quantised(x, "x")
    if out.dtype not in _DTYPES:
        raise ValueError(f"dtype {out.dtype} not supported (bfloat16 or float32)")
    _dense("x", x, (T, K), x.dtype)
    _dense("w", w, (N, K), x.dtype)
    _dense("x_scale", x_scale, (T,), torch.float32)
    _dense("w_scale", w_scale, (N,), torch.float32)
    _dense("out", out, (T, N), out.dtype)
    _on_current_device(x, x_scale, w, w_scale, out)
    if T == 0 or N == 0:
        return
    _check(load().tw_gemm_q8(
        x.data_ptr(), x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), out.data_ptr(), T, N,
        K, t0, T if t1 is None else t1, _ALL_SMS if max_sms is None else max_sms,
        _stream_handle(stream), _DTYPES[out.dtype], qt))


def _pointer(name, t, shape, dtype, dev):
    """The pointer of a tensor on device ``dev``."""
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} {dtype} tensor")
    if t.get_device() != dev:
        raise ValueError("every tensor must be on the current CUDA device")
    return t.data_ptr()


def _optional(name, t, shape, dtype, dev):
    """The pointer of a tensor that may be left out."""
    return None if t is None else _pointer(name, t, shape, dtype, dev)


def _postnorm(entry, partials, residual, weight, out, out_scale, residual_out, eps, post_weight,
              post_eps, gate, gate_tokens, block_scale, residual_scale, t0, t1, max_sms, stream):
    if residual.dim() != 2:
        raise ValueError("residual must be [T, H]")
    shape, dtype = residual.shape, residual.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"dtype {dtype} not supported (bfloat16 or float32)")
    T, H = shape
    n, n_out = len(partials), len(out)
    if not n or not n_out:
        raise ValueError("need at least one partial and one destination")
    dev = torch.cuda.current_device() if residual.is_cuda else -1
    p_arr = _pointers("partials", partials, shape, dtype, dev)
    scales, tail = (), (_DTYPES[dtype],)
    if out_scale is None:
        o_arr = _pointers("out", out, shape, dtype, dev)
    else:
        if len(out_scale) != n_out:
            raise ValueError("need a scale tensor for each destination")
        tail += (_quantised(out[0]),)
        o_arr = _pointers("out", out, shape, out[0].dtype, dev)
        scales = (_pointers("out_scale", out_scale, (T,), torch.float32, dev),)
    res = _pointer("residual", residual, shape, dtype, dev)
    res_out = _pointer("residual_out", residual_out, shape, dtype, dev)
    w = _pointer("weight", weight, (H,), dtype, dev)
    post = _optional("post_weight", post_weight, (H,), dtype, dev)
    if gate is not None and gate_tokens < 1:
        raise ValueError("gate_tokens must be at least 1")
    g = None if gate is None else _pointer("gate", gate, (-(-T // gate_tokens), H), dtype, dev)
    if dev < 0:
        raise ValueError("every tensor must be on the current CUDA device")
    if T == 0:
        return
    # (T tokens to a row of the gate and more are one row for all; more than 64 bits hold
    # would come out as another number.)
    _check(entry(p_arr, n, post, g, min(gate_tokens, T), res, w, o_arr, *scales, n_out, res_out, T, H,
                 eps if post_eps is None else post_eps, eps, block_scale, residual_scale, t0,
                 T if t1 is None else t1, _ALL_SMS if max_sms is None else max_sms,
                 _stream_handle(stream), *tail))


def tw_fused_reduce_postnorm_add_rmsnorm(partials, residual, weight, out, residual_out, eps,
                                         post_weight=None, post_eps=None, gate=None,
                                         gate_tokens=1, block_scale=1.0, residual_scale=1.0,
                                         t0=0, t1=None, max_sms=None, stream=None):
    """The fused step with a norm of the block's output (``post_weight`` [H],
    ``post_eps``: default ``eps``), its gate and scales before the residual add:
    x = residual_scale * residual + block_scale * gate * RMSNorm(sum partials).
    Without ``post_weight`` the sum is not normalised.  ``gate`` is
    [ceil(T / gate_tokens), H]: a row for every ``gate_tokens`` tokens."""
    _postnorm(load().tw_fused_reduce_postnorm_add_rmsnorm, partials, residual, weight, out, None,
              residual_out, eps, post_weight, post_eps, gate, gate_tokens, block_scale,
              residual_scale, t0, t1, max_sms, stream)


def tw_fused_reduce_postnorm_add_rmsnorm_q8(partials, residual, weight, out, out_scale,
                                            residual_out, eps, post_weight=None, post_eps=None,
                                            gate=None, gate_tokens=1, block_scale=1.0,
                                            residual_scale=1.0, t0=0, t1=None, max_sms=None,
                                            stream=None):
    """The same with ``out`` in 8 bits (int8 or float8_e4m3fn) and one scale per
    token in ``out_scale``, as in tw_fused_reduce_add_rmsnorm_q8."""
    _postnorm(load().tw_fused_reduce_postnorm_add_rmsnorm_q8, partials, residual, weight, out,
              list(out_scale), residual_out, eps, post_weight, post_eps, gate, gate_tokens,
              block_scale, residual_scale, t0, t1, max_sms, stream)


class W4Weight:
    """Weights [n, k] in 4 bits ("int4" or "e2m1") with a bf16 scale for every
    ``group`` consecutive k of a channel, in the packed form of ``include/tw.h``:
    ``packed`` (uint8) holds them.  tw_quantize_w4 fills one in, from_values takes
    a checkpoint's values and scales."""

    def __init__(self, n, k, group=128, kind="int4", device=None):
        if kind not in WTYPES:
            raise ValueError(f"kind {kind} is not one of {sorted(WTYPES)}")
        size = ctypes.c_size_t()
        _check(load().tw_w4_bytes(n, k, group, ctypes.byref(size)))
        self.n, self.k, self.group, self.kind = n, k, group, kind
        self.wtype = WTYPES[kind]
        self.packed = torch.empty(size.value, dtype=torch.uint8,
                                  device="cuda" if device is None else device)

    @classmethod
    def from_values(cls, values, scale, group=128, kind="int4"):
        """Lay out ``values`` [n, k] (of the kind's values: -8 .. 7, or 0, 0.5, 1, 1.5, 2,
        3, 4, 6 and their negatives) with ``scale`` [n, ceil(k / group)] (bf16 numbers), on
        the tensors' device.  Done with torch operations, once, when a model is loaded."""
        n, k = values.shape
        self = cls(n, k, group, kind, values.device)
        if scale.shape != (n, -(-k // group)):
            raise ValueError(f"scale must be [{n}, {-(-k // group)}]")
        held = scale.to(torch.bfloat16)
        # (A NaN stays one; bf16 infinities are numbers here, what rounds to one is not.)
        exact = scale.double()
        if not torch.all((held.double() == exact) | exact.isnan()):
            raise ValueError("scale must hold bf16 numbers")
        stripes, tiles = -(-n // 16), -(-k // 128)
        v = torch.zeros(stripes * 16, tiles * 128, dtype=torch.float32, device=values.device)
        v[:n, :k] = values
        same = values.dtype != torch.float64 or torch.equal(v[:n, :k].double(), values)
        if kind == "int4":
            code = v.round().clamp(-8, 7)
            exact, code = code, code.to(torch.int32) + 8
            fields = [(15, 4 * i, 0) for i in range(4)]
        else:
            grid = torch.tensor([0, 1, 2, 3, 4, 4, 5, 5, 6, 6, 6, 6, 7], device=v.device)
            level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=v.device)
            magnitude = grid[(v.abs() * 2).clamp(0, 12).nan_to_num().to(torch.int64)]
            exact = torch.copysign(level[magnitude], v)
            code = magnitude.to(torch.int32) + torch.signbit(v).to(torch.int32) * 8
            # Where the three low bits and the sign of a word's values go.
            fields = [(7, 6, 15), (7, 3, 12), (7, 9, 14), (7, 0, 13)]
        if not same or not torch.equal(exact, v):
            raise ValueError(f"values hold numbers that {kind} does not")
        # [stripe, half, row, tile, k / 32, k / 8 % 4, k / 2 % 4, k % 2]
        code = code.view(stripes, 2, 8, tiles, 4, 4, 4, 2)
        word = torch.zeros(code.shape[:6], dtype=torch.int32, device=v.device)
        for i, (mask, at, sign) in enumerate(fields):
            for h in range(2):
                c = code[..., i, h]
                word |= (c & mask) << (at + 16 * h)
                if kind == "e2m1":
                    word |= (c >> 3) << (sign + 16 * h)
        word = word.permute(0, 3, 1, 2, 5, 4).contiguous().view(torch.uint8)
        s = torch.zeros(stripes * 16, tiles * 128 // group, dtype=torch.bfloat16,
                        device=v.device)
        s[:n, :scale.shape[1]] = held
        s = s.view(stripes, 2, 8, tiles, 128 // group).permute(0, 3, 2, 4, 1).contiguous()
        self.packed.copy_(torch.cat([word.reshape(stripes, tiles, 1024),
                                     s.view(torch.uint8).reshape(stripes, tiles, -1)],
                                    dim=2).reshape(-1))
        return self


def _packed(w, dev):
    """The pointer of a W4Weight's packed bytes, which are those of its shape."""
    size = -(-w.n // 16) * -(-w.k // 128) * (1024 + 4096 // w.group)
    return _pointer("packed", w.packed, (size,), torch.uint8, dev)


def tw_quantize_w4(w, into, max_sms=None, stream=None):
    """Quantise ``w`` ([n, k] bfloat16 or float32) into ``into``, a W4Weight."""
    if w.dtype not in _DTYPES:
        raise ValueError(f"dtype {w.dtype} not supported (bfloat16 or float32)")
    _dense("w", w, (into.n, into.k), w.dtype)
    packed = _packed(into, w.get_device())
    _on_current_device(w)
    _check(load().tw_quantize_w4(
        w.data_ptr(), packed, into.n, into.k, into.group,
        _ALL_SMS if max_sms is None else max_sms, _stream_handle(stream), _DTYPES[w.dtype],
        into.wtype))


def tw_dequantize_w4(w, out, max_sms=None, stream=None):
    """The weights that ``w`` (a W4Weight) stands for, into ``out`` ([n, k]
    bfloat16 or float32)."""
    if out.dtype not in _DTYPES:
        raise ValueError(f"dtype {out.dtype} not supported (bfloat16 or float32)")
    _dense("out", out, (w.n, w.k), out.dtype)
    packed = _packed(w, out.get_device())
    _on_current_device(out)
    _check(load().tw_dequantize_w4(
        packed, out.data_ptr(), w.n, w.k, w.group,
        _ALL_SMS if max_sms is None else max_sms, _stream_handle(stream), _DTYPES[out.dtype],
        w.wtype))


def tw_gemm_w4(x, w, out, x_scale=None, t0=0, t1=None, max_sms=None, stream=None):
    """out[t, n] = sum_k x[t, k] * w[n, k] on rows [t0, t1): ``x`` [T, k] bfloat16
    or float32, or int8 or float8_e4m3fn with ``x_scale`` [T]; ``w`` a W4Weight;
    ``out`` [T, n] bfloat16 or float32."""
    shape = x.shape
    if len(shape) != 2 or shape[1] != w.k:
        raise ValueError(f"x must be [T, {w.k}]")
    T = shape[0]
    xt, dt = _XTYPES.get(x.dtype), _DTYPES.get(out.dtype)
    if xt is None or dt is None:
        raise ValueError(f"dtypes {x.dtype}, {out.dtype} not supported")
    if (x_scale is None) != (xt < 2):
        raise ValueError("x_scale goes with 8-bit x, and only with it")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    dev = torch.cuda.current_device() if x.is_cuda else -1
    to = _pointer("out", out, (T, w.n), out.dtype, dev)
    packed = _packed(w, dev)
    if dev < 0 or x.get_device() != dev:
        raise ValueError("every tensor must be on the current CUDA device")
    scale = _optional("x_scale", x_scale, (T,), torch.float32, dev)
    if T == 0:
        return
    _check(load().tw_gemm_w4(
        x.data_ptr(), scale, packed, to, T, w.n, w.k, w.group, t0,
        T if t1 is None else t1, _ALL_SMS if max_sms is None else max_sms,
        _stream_handle(stream), xt, dt, w.wtype))


def tw_split_launch(partials, residual, weight, out, residual_out, eps,
                    t_split=-1, max_sms=None, s0=None, s1=None):
    """Two-chunk token split: rows [0, t_split) on s0, [t_split, T) on s1.
    Synchronising s0 covers both chunks."""
    p_arr, n, o_arr, n_out, T, H, dt = _marshal(partials, residual, weight,
                                                out, residual_out)
    if s1 is None:
        raise ValueError("tw_split_launch needs a second stream s1")
    rc = load().tw_split_launch(
        p_arr, n, residual.data_ptr(), weight.data_ptr(), o_arr, n_out,
        residual_out.data_ptr(), T, H, eps, t_split,
        _ALL_SMS if max_sms is None else max_sms, _stream_handle(s0),
        _stream_handle(s1), dt)
    _check(rc)


def tw_host_workspace_bytes(n_parts, n_out, H, chunk_tokens, dtype):
    """Device workspace bytes of tw_fused_reduce_add_rmsnorm_host."""
    out = ctypes.c_size_t()
    _check(load().tw_host_workspace_bytes(n_parts, n_out, H, chunk_tokens,
                                          _DTYPES[dtype], ctypes.byref(out)))
    return out.value


def tw_fused_reduce_add_rmsnorm_host(partials, residual, weight, out,
                                     residual_out, eps, workspace, chunk_tokens,
                                     t0=0, t1=None, max_sms=None, stream=None):
    """The fused step on pinned HOST tensors.  ``chunk_tokens`` >= 1: pipelined
    in chunks of that many tokens through the device ``workspace`` (a uint8
    CUDA tensor of at least tw_host_workspace_bytes bytes).  ``chunk_tokens``
    == 0: one kernel reads the host tensors in place (``workspace`` may be
    None)."""
    p_arr, n, o_arr, n_out, T, H, dt = _marshal(partials, residual, weight,
                                                out, residual_out, on_device=False)
    if workspace is not None and not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    rc = load().tw_fused_reduce_add_rmsnorm_host(
        p_arr, n, residual.data_ptr(), weight.data_ptr(), o_arr, n_out,
        residual_out.data_ptr(), T, H, eps, t0, T if t1 is None else t1,
        _ALL_SMS if max_sms is None else max_sms,
        None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        chunk_tokens, _stream_handle(stream), dt)
    _check(rc)


def tw_fused_reduce_add_rmsnorm_host_noalloc(partials, residual, weight, out,
                                             residual_out, eps, chunk_tokens=0,
                                             t0=0, t1=None, max_sms=None,
                                             stream=None):
    """The host-buffer step for callers that cannot allocate device memory:
    pinned host tensors only; the library stages the chunks in its own
    fixed device array (chunk_tokens <= 0: the largest chunk that fits)."""
    p_arr, n, o_arr, n_out, T, H, dt = _marshal(partials, residual, weight,
                                                out, residual_out, on_device=False)
    rc = load().tw_fused_reduce_add_rmsnorm_host_noalloc(p_arr, n, residual.data_ptr(), weight.data_ptr(), o_arr, n_out,
            residual_out.data_ptr(), T, H, eps, t0, T if t1 is None else t1,
            _ALL_SMS if max_sms is None else max_sms, chunk_tokens,
            _stream_handle(stream), dt)
    _check(rc)


def tw_device_status(clear=False):
    """Device status word: nonzero if a kernel gave up on a bounded wait."""
    rc = load().tw_device_status(1 if clear else 0)
    if rc < 0:
        raise TwError(-4, load().tw_last_error_string().decode())
    return rc


def tw_last_error_string():
    return load().tw_last_error_string().decode()


def tw_version():
    return load().tw_version()


class Prepared:
    """A tw_fused_reduce_add_rmsnorm_ex call with its arguments marshalled
    once, for launch loops where per-call Python work would outlast the
    kernel.  The tensors must stay alive and unchanged in shape."""

    def __init__(self, partials, residual, weight, out, residual_out, eps, t0=0,
                 t1=None, max_sms=None, path="auto", ready=None, block_tokens=0, epoch=0):
        p_arr, n, o_arr, n_out, T, H, dt = _marshal(partials, residual, weight,
                                                    out, residual_out)
        self._keep = (p_arr, o_arr, list(partials), residual, weight, list(out),
                      residual_out)
        self._args = [p_arr, n, residual.data_ptr(), weight.data_ptr(), o_arr,
                      n_out, residual_out.data_ptr(), T, H, eps, t0,
                      T if t1 is None else t1,
                      _ALL_SMS if max_sms is None else max_sms]
        if ready is not None:
            # tw_fused_reduce_add_rmsnorm_flags: gated by readiness flags.
            if ready.dtype != torch.int32 or not ready.is_cuda:
                raise ValueError("ready must be an int32 CUDA tensor")
            self._keep += (ready,)
            self._fn = load().tw_fused_reduce_add_rmsnorm_flags
            self._tail = [dt, ready.data_ptr(), block_tokens, epoch & 0xFFFFFFFF]
        elif path == "colsplit":
            # tw_fused_reduce_add_rmsnorm_colsplit: zero-padded column split.
            self._fn = load().tw_fused_reduce_add_rmsnorm_colsplit
            self._tail = [dt]
        else:
            self._fn = load().tw_fused_reduce_add_rmsnorm_ex
            self._tail = [dt, PATHS[path], None]

    def __call__(self, stream_handle):
        """Launch on the raw cudaStream_t handle (an int)."""
        rc = self._fn(*self._args, stream_handle, *self._tail)
        if rc != 0:
            _check(rc)


def prepare(partials, residual, weight, out, residual_out, eps, t0=0, t1=None,
            max_sms=None, path="auto", ready=None, block_tokens=0, epoch=0):
    """Marshal a fused call once; returns a :class:`Prepared` callable.
    ``path`` is a kernel name of tw_fused_reduce_add_rmsnorm_ex, or "colsplit"
    for tw_fused_reduce_add_rmsnorm_colsplit; with ``ready`` the call is
    tw_fused_reduce_add_rmsnorm_flags."""
    return Prepared(partials, residual, weight, out, residual_out, eps, t0, t1,
                    max_sms, path, ready, block_tokens, epoch)
