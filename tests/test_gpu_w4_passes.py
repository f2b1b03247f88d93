"""The 4-bit product where a cluster's CTAs use the room for their sums again and again:
several passes over the channels, several blocks of tokens, slices of K."""
import pytest
import torch

from tests.test_gpu_w4_gemm import check, make, make_x
from reduce_residual_rmsnorm_tw_gb300 import tw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,n,k,group,kind,xtype,max_sms", [
    # (CTAs of a cluster, passes, blocks of tokens:)
    (64, 3000, 8192, 64, "int4", "bf16", 16),    # 4, 2, 2
    (64, 3000, 8192, 64, "int4", "bf16", 8),     # 4, 4, 2
    (64, 3000, 16384, 64, "e2m1", "int8", 24),   # 8, 4, 2
    (12, 9000, 65536, 32, "int4", "f32", 40),    # 8, 8, 4
    (3, 2000, 65536, 32, "int4", "f32", 8),      # 8, 8, 1
    (2, 2000, 65536, 32, "int4", "f32", 2),      # 2, 2, 2, four slices of K
    (100, 9000, 28672, 128, "int4", "bf16", 1 << 20),
    (70, 20000, 8192, 128, "e2m1", "bf16", 1 << 20)])
def test_passes_and_blocks_give_equal_bits_every_time(t, n, k, group, kind, xtype, max_sms):
    w4, w64 = make(n, k, group, kind)
    x, scale, x64 = make_x(t, k, xtype)
    first = torch.zeros(t, n, device="cuda")
    tw.tw_gemm_w4(x, w4, first, x_scale=scale, max_sms=max_sms)
    check(first, x64, w64, group, xtype == "f32")
    outs = [torch.zeros_like(first) for _ in range(8)]
    for out in outs:
        tw.tw_gemm_w4(x, w4, out, x_scale=scale, max_sms=max_sms)
    torch.cuda.synchronize()
    assert all(torch.equal(out, first) for out in outs)
    assert tw.tw_device_status() == 0
