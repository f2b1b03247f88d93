"""The fused step with 8-bit outputs and the row quantisation against 64-bit
references."""
import numpy as np
import pytest
import torch

import oracle
from reduce_residual_rmsnorm_tw_gb300 import inputs, tw
from reduce_residual_rmsnorm_tw_gb300.inputs import Workload
from tests.parity import SENTINEL, check_close
from tests.q8_reference import KIND, U, check_rows, f64, row_error

pytestmark = pytest.mark.gpu


def empty_outputs(wl, quant):
    # 77 is a valid int8 and e4m3 byte; the scale sentinel is never a scale.
    q = [torch.full((wl.T, wl.H), 77, dtype=torch.uint8, device="cuda").view(KIND[quant])
         for _ in range(wl.n_out)]
    s = [torch.full((wl.T,), -3.0, device="cuda") for _ in range(wl.n_out)]
    return q, s, torch.full((wl.T, wl.H), SENTINEL, dtype=wl.torch_dtype, device="cuda")


def check_norm(wl, quant, t0=0, t1=None, max_sms=None, in_place=False):
    t1 = wl.T if t1 is None else t1
    host = inputs.make_inputs(wl)
    parts, res = [p.cuda() for p in host["partials"]], host["residual"].cuda()
    q, s, res_out = empty_outputs(wl, quant)
    if in_place:
        res_out = res
    tw.tw_fused_reduce_add_rmsnorm_q8(parts, res, host["weight"].cuda(), q, s, res_out, wl.eps,
                                      t0, t1, max_sms=max_sms)
    torch.cuda.synchronize()
    p64 = [inputs.to_f64(p) for p in host["partials"]]
    r64, w64 = inputs.to_f64(host["residual"]), inputs.to_f64(host["weight"])
    ref, ref_res = oracle.reordered(p64, r64, w64, wl.eps, n_out=1, t0=t0, t1=t1)
    rows = slice(t0, t1)
    x = sum(p64) + r64
    # The row's values: the sum's error; weight and scale multiplies, the
    # division and the inverse rms (a sum of H squares kept as at most 64
    # terms in a chain, then by tree, and rsqrtf's 2 ulp).
    rel = 2 * row_error([(p * w64)[rows] for p in p64 + [r64]], (x * w64)[rows]) + 100 * U
    for k in range(wl.n_out):
        check_rows(q[k][rows], s[k][rows], ref[0][rows], quant, rel, f"{wl.name} out[{k}]")
        assert torch.equal(q[k].view(torch.uint8), q[0].view(torch.uint8))
        assert torch.equal(s[k], s[0])
        outside = torch.cat([q[k].view(torch.uint8)[:t0], q[k].view(torch.uint8)[t1:]])
        assert bool((outside == 77).all()) and bool((s[k][:t0] == -3).all()) and \
            bool((s[k][t1:] == -3).all())
    check_close(res_out[rows], ref_res[rows], wl.dtype, f"{wl.name} residual_out")
    if not in_place:
        assert bool((torch.cat([res_out[:t0], res_out[t1:]]).float() == SENTINEL).all())
    return q, s, res_out


# Rows of one vector up to the largest, a row that leaves threads idle; one
# token, both sides of the cluster kernel's 128 tokens, units of 2 and 4
# tokens, launches long enough to claim units (16 per CTA).
NORMS = [(8, 1, 8192, "bf16", 1), (3, 7, 8, "bf16", 2), (8, 64, 8192, "bf16", 1),
         (1, 128, 1000, "bf16", 1), (16, 129, 4104, "bf16", 8), (2, 2048, 4096, "bf16", 1),
         (5, 33, 16384, "bf16", 2), (4, 301, 5120, "f32", 4), (2, 5, 4, "f32", 1),
         (2, 19, 8192, "f32", 1), (2, 10100, 512, "bf16", 1), (1, 5000, 1024, "f32", 1)]


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("parts,T,H,dtype,outs", NORMS)
def test_norm_matches_oracle(parts, T, H, dtype, outs, quant):
    check_norm(Workload(f"q8_{parts}_{T}_{H}_{dtype}", parts, T, H, dtype, 1e-5, outs, 71), quant)
    assert tw.tw_device_status() == 0


@pytest.mark.parametrize("max_sms", [1, 2, 9, None])
def test_norm_ranges_budgets_and_in_place(max_sms):
    # The same bits for every budget and split of the tokens, nothing outside
    # the range written.
    wl = Workload("q8_ranges", 4, 300, 4096, "bf16", 1e-6, 1, 72)
    q0, s0, r0 = check_norm(wl, "int8", max_sms=max_sms, in_place=True)
    q1, s1, r1 = check_norm(wl, "int8", 3, 297, max_sms=max_sms)
    assert torch.equal(q0[0][3:297], q1[0][3:297]) and torch.equal(r0[3:297], r1[3:297])
    q2, s2, _ = check_norm(wl, "int8", 295, 296)
    assert torch.equal(q0[0][295], q2[0][295])
    assert torch.allclose(s0[0][295], s2[0][295], rtol=20 * U)  # another kernel's sum order


def test_norm_residual_is_the_plain_steps():
    # residual_out is bit for bit the unquantised entry point's.
    wl = Workload("q8_res", 8, 200, 8192, "bf16", 1e-6, 1, 73)
    d = inputs.make_inputs(wl, device="cuda")
    q, s, r = empty_outputs(wl, "e4m3")
    tw.tw_fused_reduce_add_rmsnorm_q8(d["partials"], d["residual"], d["weight"], q, s, r, wl.eps)
    o, r2 = torch.empty_like(r), torch.empty_like(r)
    tw.tw_fused_reduce_add_rmsnorm(d["partials"], d["residual"], d["weight"], [o], r2, wl.eps)
    assert torch.equal(r, r2)


SPECIAL = [0.0, float("nan"), float("inf"), float("-inf"), 1e-37]


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("T", [6, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_and_non_finite_rows(dtype, T, quant):
    # Row i % 6 < 5 is all zeros but for one special value (or is zero):
    # zero and tiny rows get scale 0 and zeros, the others scale NaN and
    # zeros; the sixth kind is an ordinary row next to them.
    H = 1024
    x = torch.zeros(T, H, dtype=torch.float32)
    for t in range(T):
        if t % 6 < 5:
            x[t, 700] = SPECIAL[t % 6]
        else:
            x[t] = torch.linspace(-1, 1, H)
    x = x.to(inputs.DTYPES[dtype]).cuda()
    zero = torch.zeros_like(x)
    w = torch.ones(H, dtype=x.dtype, device="cuda")
    for op in ("norm", "rows"):
        q = torch.full((T, H), 77, dtype=torch.uint8, device="cuda").view(KIND[quant])
        s = torch.full((T,), -3.0, device="cuda")
        if op == "norm":
            tw.tw_fused_reduce_add_rmsnorm_q8([x], zero, w, [q], [s], torch.empty_like(x), 1e-5)
        else:
            tw.tw_quantize_rows_q8(x, q, s)
        g, sc = f64(q), f64(s)
        for t in range(T):
            kind = t % 6
            if kind == 5:
                assert np.abs(g[t]).max() == {"int8": 127, "e4m3": 448}[quant] and sc[t] > 0
            else:
                assert (g[t] == 0).all(), (op, t)
                assert np.isnan(sc[t]) if kind in (1, 2, 3) else sc[t] == 0, (op, t, sc[t])


ROWS = [(1, 8192, "bf16"), (37, 1000, "bf16"), (4096, 256, "bf16"), (300, 8, "bf16"),
        (77, 264, "bf16"), (9, 520, "bf16"), (200, 1032, "bf16"), (150, 2056, "bf16"),
        (3, 16384, "bf16"), (2500, 4, "f32"), (1, 4, "f32"), (31, 8192, "f32"),
        (513, 1236, "f32")]


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("T,H,dtype", ROWS)
def test_quantize_matches_reference(T, H, dtype, quant):
    g = torch.Generator()
    g.manual_seed(T * H)
    x = torch.randn(T, H, generator=g).to(inputs.DTYPES[dtype])
    x *= torch.logspace(-6, 6, T)[:, None].to(x.dtype)  # rows of every size
    t0, t1 = (0, T) if T < 3 else (1, T - 1)
    for max_sms in (None, 3):
        q = torch.full((T, H), 77, dtype=torch.uint8, device="cuda").view(KIND[quant])
        s = torch.full((T,), -3.0, device="cuda")
        tw.tw_quantize_rows_q8(x.cuda(), q, s, t0, t1, max_sms=max_sms)
        # One division for the scale, one for the factor, one multiply.
        check_rows(q[t0:t1], s[t0:t1], inputs.to_f64(x[t0:t1]), quant,
                   np.full(t1 - t0, 3 * U), f"rows {T} {H} {dtype}")
        b = q.view(torch.uint8)
        assert bool((torch.cat([b[:t0], b[t1:]]) == 77).all())
        assert bool((torch.cat([s[:t0], s[t1:]]) == -3).all())


def test_empty_batches_and_other_streams():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    tw.tw_quantize_rows_q8(x, torch.empty(0, 64, dtype=torch.int8, device="cuda"),
                           torch.empty(0, device="cuda"))
    side = torch.cuda.Stream()
    x = torch.randn(500, 512, device="cuda").bfloat16()
    a, b = (torch.zeros(500, 512, dtype=torch.int8, device="cuda") for _ in range(2))
    sa, sb = (torch.zeros(500, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    tw.tw_quantize_rows_q8(x, a, sa)
    tw.tw_quantize_rows_q8(x, b, sb, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(sa, sb)


def test_offsets_past_2_to_31():
    # 2.3e9 elements a tensor; the last rows against the reference.
    T, H = 140000, 16384
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_()
    q = torch.zeros(T, H, dtype=torch.int8, device="cuda")
    s = torch.zeros(T, device="cuda")
    tw.tw_quantize_rows_q8(x, q, s)
    last = slice(T - 3, T)
    check_rows(q[last], s[last], inputs.to_f64(x[last]), "int8", np.full(3, 3 * U), "rows")
    q.zero_()
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    r = torch.empty_like(x)
    tw.tw_fused_reduce_add_rmsnorm_q8([x], x, w, [q], [s], r, 1e-5)
    v = 2 * inputs.to_f64(x[last])
    ref = v / np.sqrt((v ** 2).mean(axis=1, keepdims=True) + 1e-5)
    check_rows(q[last], s[last], ref, "int8", np.full(3, 100 * U), "norm")
    assert torch.equal(r[last], 2 * x[last])  # exact in bf16
