"""The joined step's two ways to multiply refuse the same calls: below the number of tokens
from which the weights are read back for a library product, and from there on."""
import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import layer_step, tw

pytestmark = pytest.mark.gpu
H, K = 256, 512


@pytest.mark.parametrize("T", [32, 33])
@pytest.mark.parametrize("wrong", [
    "x_scale", "rows of partial 0", "features of partial 0", "transposed partial 0",
    "features of x", "transposed x", "shape of workspace", "type of workspace",
    "transposed workspace", "workspace on the host", "x over partial 0"])
def test_refusals_on_both_sides(T, wrong):
    assert layer_step.w4_library_tokens(H, K) == 33
    bf = dict(dtype=torch.bfloat16, device="cuda")
    w4 = tw.W4Weight(H, K, 64, "int4")
    tw.tw_quantize_w4(torch.randn(H, K, device="cuda"), w4)
    x, partial = torch.randn(T, K, **bf), torch.full((T, H), 3.0, **bf)
    residual, out, res = torch.randn(T, H, **bf), torch.zeros(T, H, **bf), torch.zeros(T, H, **bf)
    weight, workspace, extra = torch.rand(H, **bf), torch.full((H, K), 7.0, **bf), {}
    if wrong == "x_scale":
        extra["x_scale"] = torch.rand(T, device="cuda")
    elif wrong == "rows of partial 0":
        partial = torch.full((T + 1, H), 3.0, **bf)
    elif wrong == "features of partial 0":
        partial = torch.full((T, H // 2), 3.0, **bf)
    elif wrong == "transposed partial 0":
        partial = torch.full((H, T), 3.0, **bf).t()
    elif wrong == "features of x":
        x = torch.randn(T, K + 16, **bf)
    elif wrong == "transposed x":
        x = torch.randn(K, T, **bf).t()
    elif wrong == "shape of workspace":
        workspace = torch.full((H, K + 16), 7.0, **bf)
    elif wrong == "type of workspace":
        workspace = workspace.float()
    elif wrong == "transposed workspace":
        workspace = torch.full((K, H), 7.0, **bf).t()
    elif wrong == "workspace on the host":
        workspace = workspace.cpu()
    elif wrong == "x over partial 0":
        both = torch.full((T, K), 3.0, **bf)
        x, partial = both, both.view(-1)[:T * H].view(T, H)
    shape = partial.shape
    with pytest.raises((ValueError, tw.TwError)):
        layer_step.sandwich_layer_step_w4(x, w4, [partial], residual, weight, [out], res, 1e-5,
                                          workspace=workspace, post_weight=weight, **extra)
    torch.cuda.synchronize()
    # Nothing was launched, and no tensor resized.
    assert partial.shape == shape and torch.all(partial == 3)
    assert torch.all(workspace == 7) and not out.any() and not res.any()
