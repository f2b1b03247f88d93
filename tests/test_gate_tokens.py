"""Tokens to a row of the gate beyond what 64 bits hold: one row for all, as documented."""
import ctypes

import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import tw

SIZES = [5, 6, 2 ** 31, 2 ** 63 - 1, 2 ** 63, 2 ** 64, 2 ** 64 + 1, 10 ** 30]


@pytest.mark.parametrize("gate_tokens", SIZES)
def test_what_the_library_is_given(monkeypatch, gate_tokens):
    """The number that arrives behind the binding, on the CPU (the entry point a stand-in
    that takes it as C does)."""
    given = []

    def entry(p_arr, n, post, gate, tokens, *rest):
        given.append(ctypes.c_int64(tokens).value)
        return 0
    monkeypatch.setattr(tw, "_stream_handle", lambda stream: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(tw, "_pointers", lambda *args: None)
    monkeypatch.setattr(tw, "_pointer", lambda *args: None)

    class Residual:  # a [5, 64] tensor on device 0
        is_cuda, dtype, shape = True, torch.bfloat16, torch.Size([5, 64])

        def dim(self):
            return 2
    gate = torch.zeros(1, 64, dtype=torch.bfloat16)
    tw._postnorm(entry, [0], Residual(), 0, [0], None, 0, 1e-6, None, None, gate, gate_tokens, 1.0,
                 1.0, 0, None, None, None)
    assert given == [5]


@pytest.mark.gpu
@pytest.mark.parametrize("gate_tokens", SIZES)
def test_one_row_for_all(gate_tokens):
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()
    parts, residual, gate, weight = [normal(5, 512)], normal(5, 512), normal(1, 512), normal(512)
    got = []
    for tokens, rows in ((gate_tokens, gate), (1, gate.expand(5, 512).contiguous())):
        out, res = torch.zeros_like(residual), torch.zeros_like(residual)
        tw.tw_fused_reduce_postnorm_add_rmsnorm(parts, residual, weight, [out], res, 1e-6, gate=rows,
                                                gate_tokens=tokens)
        got.append((out, res))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
