"""The step with two norms where an SM budget makes a token's cluster smaller: two, four
and eight CTAs, one to four vectors of the row to a thread."""
import pytest

from tests.test_gpu_postnorm import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("quant", [None, "int8", "e4m3"])
@pytest.mark.parametrize("H,dtype", [(8192, "bf16"), (16384, "bf16"), (8192, "f32"), (4104, "bf16"),
                                     (2052, "f32"), (12296, "bf16")])
@pytest.mark.parametrize("max_sms", [1, 2, 3, 4, 7, 8])
def test_one_token(max_sms, H, dtype, quant):
    check(3, 1, H, dtype, gate_tokens=1, max_sms=max_sms, quant=quant, n_out=2, block_scale=0.5)
    check(2, 1, H, dtype, post=False, max_sms=max_sms, quant=quant, in_place=True)


@pytest.mark.parametrize("quant", [None, "int8"])
@pytest.mark.parametrize("T,max_sms", [(2, 16), (3, 31), (4, 32), (9, 76), (1, 152), (18, 151)])
def test_several_tokens(T, max_sms, quant):
    check(4, T + 2, 8192, "bf16", gate_tokens=2, max_sms=max_sms, quant=quant, t0=1, t1=T + 1)
    check(9, T + 2, 8192, "f32", max_sms=max_sms, quant=quant, t0=1, t1=T + 1, residual_scale=1.4)
