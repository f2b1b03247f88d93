"""What a checkpoint's values and scales must be to be laid out, on the CPU."""
import numpy as np
import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import build as twbuild
from reduce_residual_rmsnorm_tw_gb300 import tw
from tests import w4_reference as ref


@pytest.fixture(scope="module", autouse=True)
def lib():
    twbuild.build()
    return tw.load()


@pytest.mark.parametrize("kind", ["int4", "e2m1"])
@pytest.mark.parametrize("value,dtype", [
    # Finite numbers that round to an infinity, numbers that lose bits on the way to fp32.
    (torch.finfo(torch.float32).max, torch.float32), (-3.4e38, torch.float32),
    (3.3961e38, torch.float32), (1.0 + 2.0 ** -40, torch.float64), (1e39, torch.float64),
    (2.0 ** -150, torch.float64), (2.0 ** -134, torch.float32)])
def test_scales_that_are_not_bf16_are_refused(value, dtype, kind):
    v, s = torch.ones(8, 64), torch.ones(8, 2, dtype=dtype)
    s[3, 1] = value
    with pytest.raises(ValueError):
        tw.W4Weight.from_values(v, s, 32, kind)


@pytest.mark.parametrize("kind", ["int4", "e2m1"])
def test_values_that_lose_bits_on_the_way_are_refused(kind):
    v, s = torch.ones(8, 64, dtype=torch.float64), torch.ones(8, 2)
    assert np.all(ref.unpack(tw.W4Weight.from_values(v, s, 32, kind))[0] == 1)
    for value in (1.0 + 2.0 ** -40, 2.0 ** -150, -4.0 - 2.0 ** -45):
        v[2, 9] = value
        with pytest.raises(ValueError):
            tw.W4Weight.from_values(v, s, 32, kind)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float64])
def test_every_bf16_scale_is_taken(dtype):
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    s = bits.view(torch.bfloat16).view(1024, 64)
    w4 = tw.W4Weight.from_values(torch.ones(1024, 64 * 32), s.to(dtype), 32, "int4")
    got = torch.from_numpy(ref.unpack(w4)[1])
    assert torch.equal(got.nan_to_num(nan=7.0, posinf=1e300, neginf=-1e300),
                       s.double().nan_to_num(nan=7.0, posinf=1e300, neginf=-1e300))


@pytest.mark.parametrize("dtype", [torch.float16, torch.int32, torch.float8_e4m3fn,
                                   torch.float8_e5m2])
def test_scales_of_other_types(dtype):
    s = torch.tensor([0.0, 1.0, 2.0, 4.0, 16.0, -8.0, 64.0, 128.0]).view(4, 2)
    got = ref.unpack(tw.W4Weight.from_values(torch.ones(4, 64), s.to(dtype), 32, "int4"))[1]
    assert np.array_equal(got, s.double().numpy())


@pytest.mark.parametrize("dtype", [torch.int8, torch.int64, torch.float16, torch.float64])
def test_values_of_any_type(dtype):
    v = torch.arange(-8, 8).repeat(8, 4).to(dtype)
    w4 = tw.W4Weight.from_values(v, torch.ones(8, 2), 32, "int4")
    assert np.array_equal(ref.unpack(w4)[0], v.double().numpy())
