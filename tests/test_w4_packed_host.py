"""A W4Weight whose packed bytes are not those of its shape is refused by the binding, by
name and before anything else could read past them, on the CPU."""
import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import build as twbuild
from reduce_residual_rmsnorm_tw_gb300 import tw


@pytest.fixture(scope="module", autouse=True)
def lib():
    twbuild.build()
    return tw.load()


def calls(w4):
    n, k = w4.n, w4.k
    rows = torch.zeros(n, k, dtype=torch.bfloat16)
    return [lambda: tw.tw_quantize_w4(rows, w4), lambda: tw.tw_dequantize_w4(w4, rows),
            lambda: tw.tw_gemm_w4(torch.zeros(3, k), w4, torch.zeros(3, n))]


@pytest.mark.parametrize("change", ["short", "long", "none", "type", "stride", "more channels",
                                    "longer rows", "finer groups"])
def test_packed_of_another_size(change):
    w4 = tw.W4Weight(40, 256, 128, "int4", "cpu")
    packed = w4.packed
    if change == "short":
        w4.packed = packed[:-16]
    elif change == "long":
        w4.packed = torch.zeros(packed.numel() + 16, dtype=torch.uint8)
    elif change == "none":
        w4.packed = packed[:0]
    elif change == "type":
        w4.packed = packed.view(torch.int8)
    elif change == "stride":
        w4.packed = torch.zeros(2 * packed.numel(), dtype=torch.uint8)[::2]
    elif change == "more channels":
        w4.n = 56
    elif change == "longer rows":
        w4.k = 400
    else:
        w4.group = 32
    for call in calls(w4):
        with pytest.raises(ValueError, match="packed must be"):
            call()


@pytest.mark.parametrize("n,k,group", [(1, 16, 32), (16, 128, 64), (17, 144, 128)])
def test_its_own_size_is_not_refused(n, k, group):
    for call in calls(tw.W4Weight(n, k, group, "e2m1", "cpu")):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
