"""The stream of a call without one: torch's current stream, with and without the
private call that gives its handle."""
import types

import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import tw


def test_without_the_private_call(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(tw, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda: types.SimpleNamespace(cuda_stream=1234))
    assert tw._stream_handle(None) == 1234


def test_given_streams_pass_through():
    assert tw._stream_handle(77) == 77
    assert tw._stream_handle(types.SimpleNamespace(cuda_stream=88)) == 88


@pytest.mark.gpu
@pytest.mark.parametrize("private", [True, False])
def test_calls_run_on_the_current_stream(monkeypatch, private):
    if not private:
        monkeypatch.setattr(tw, "_raw_stream", None)
    side = torch.cuda.Stream()
    assert tw._stream_handle(None) == torch.cuda.current_stream().cuda_stream
    x = torch.randn(300, 512, device="cuda").bfloat16()
    q, s = torch.zeros(300, 512, dtype=torch.int8, device="cuda"), torch.zeros(300, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert tw._stream_handle(None) == side.cuda_stream
        tw.tw_quantize_rows_q8(x, q, s)
    side.synchronize()
    assert bool((q.abs().amax(1) == 127).all()) and bool((s > 0).all())
