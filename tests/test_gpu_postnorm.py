"""The step with two norms, gate and scales against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import inputs, tw
from tests.postnorm_reference import step
from tests.q8_reference import KIND, check_rows, f64

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def make(n_parts, T, H, dtype, post=True, gate_tokens=None, seed=0):
    g = torch.Generator().manual_seed(seed + 1000 * T + H + n_parts)
    kind = DTYPES[dtype]

    def normal(*shape):
        return torch.randn(*shape, generator=g).to(kind)
    host = {"partials": [normal(T, H) for _ in range(n_parts)], "residual": normal(T, H),
            "weight": (torch.rand(H, generator=g) + 0.5).to(kind)}
    block = {"post_weight": (torch.rand(H, generator=g) + 0.5).to(kind) if post else None,
             "gate": None if gate_tokens is None else normal(-(-T // gate_tokens), H)}
    return host, block


def on_gpu(host, block):
    d = {k: [p.cuda() for p in v] if k == "partials" else v.cuda() for k, v in host.items()}
    return d, {k: None if v is None else v.cuda() for k, v in block.items()}


def expected(host, block, **kwargs):
    d64 = {k: [f64(p) for p in v] if k == "partials" else f64(v) for k, v in host.items()}
    b64 = {k: None if v is None else f64(v) for k, v in block.items()}
    return step(d64, **b64, **kwargs)


def close(got, want, err, what):
    half = torch.finfo(got.dtype).eps / 2
    g = f64(got)
    bound = err + half * (np.abs(want) + err)
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} off, worst {np.max(np.abs(g - want) / bound)}"


def check(n_parts, T, H, dtype, post=True, gate_tokens=None, n_out=1, t0=0, t1=None, max_sms=None,
          quant=None, seed=0, in_place=False, **scales):
    host, block = make(n_parts, T, H, dtype, post, gate_tokens, seed)
    d, b = on_gpu(host, block)
    t1 = T if t1 is None else t1
    kwargs = {"gate_tokens": gate_tokens or 1, **scales}
    x, y, ex, ey = expected(host, block, eps=EPS, **kwargs)
    rows = slice(t0, t1)
    res_out = d["residual"] if in_place else torch.full_like(d["residual"], 7.0)
    args = dict(post_weight=b["post_weight"], gate=b["gate"], t0=t0, t1=t1, max_sms=max_sms, **kwargs)
    what = (n_parts, T, H, dtype, post, gate_tokens, quant)
    if quant is None:
        out = [torch.full_like(d["residual"], 7.0) for _ in range(n_out)]
        tw.tw_fused_reduce_postnorm_add_rmsnorm(d["partials"], d["residual"], d["weight"], out,
                                                res_out, EPS, **args)
        for o in out:
            close(o[rows], y[rows], ey[rows], what)
            assert torch.all(o[:t0] == 7) and torch.all(o[t1:] == 7)
    else:
        out = [torch.full((T, H), 1.0, device="cuda").to(KIND[quant]) for _ in range(n_out)]
        scale = [torch.full((T,), 7.0, device="cuda") for _ in range(n_out)]
        tw.tw_fused_reduce_postnorm_add_rmsnorm_q8(d["partials"], d["residual"], d["weight"], out,
                                                   scale, res_out, EPS, **args)
        # The norm's quotients may go to either side within 2 ulp of a middle.
        rel = ey.max(axis=1) / np.abs(y).max(axis=1) + 6 * 2.0 ** -24
        for o, s in zip(out, scale):
            check_rows(o[rows], s[rows], y[rows], quant, rel[rows], what)
            assert torch.all(s[:t0] == 7) and torch.all(s[t1:] == 7)
            assert torch.all(o[:t0].float() == 1) and torch.all(o[t1:].float() == 1)
    close(res_out[rows], x[rows], ex[rows], what)
    if not in_place:
        assert torch.all(res_out[:t0] == 7) and torch.all(res_out[t1:] == 7)
    else:
        rest = torch.ones(T, dtype=torch.bool)
        rest[rows] = False
        assert torch.equal(res_out.cpu()[rest], host["residual"][rest])


SHAPES = [(1, 1, 8, "bf16"), (2, 3, 64, "bf16"), (8, 1, 8192, "bf16"), (3, 5, 264, "bf16"),
          (8, 64, 8192, "bf16"), (2, 300, 4096, "bf16"), (4, 37, 1000, "bf16"),
          (1, 200, 512, "bf16"), (16, 70, 2048, "bf16"), (5, 150, 16384, "bf16"),
          (1, 1, 4, "f32"), (4, 90, 5120, "f32"), (3, 2, 8192, "f32"), (2, 1000, 100, "f32"),
          (7, 77, 1028, "f32"), (2, 400, 8192, "f32"), (9, 129, 260, "f32")]


@pytest.mark.parametrize("quant", [None, "int8", "e4m3"])
@pytest.mark.parametrize("n_parts,T,H,dtype", SHAPES)
def test_shapes(n_parts, T, H, dtype, quant):
    check(n_parts, T, H, dtype, quant=quant, n_out=1 + T % 2)


@pytest.mark.parametrize("quant", [None, "int8"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate_tokens", [None, 1, 3, 50, 10 ** 12])
@pytest.mark.parametrize("T,H,dtype", [(2, 8192, "bf16"), (101, 136, "bf16"), (130, 5120, "f32")])
def test_gates_and_scales(T, H, dtype, gate_tokens, post, quant):
    check(3, T, H, dtype, post, gate_tokens, quant=quant, block_scale=0.22, residual_scale=-1.4)


@pytest.mark.parametrize("max_sms", [1, 2, 5, 8, 100, 152])
@pytest.mark.parametrize("T,H,dtype", [(3, 8192, "bf16"), (70, 4096, "bf16"), (33, 200, "f32"),
                                       (20, 8192, "f32")])
def test_budgets(T, H, dtype, max_sms):
    check(2, T, H, dtype, gate_tokens=1, max_sms=max_sms)


@pytest.mark.parametrize("quant", [None, "int8"])
@pytest.mark.parametrize("n_parts,T,H,dtype,max_sms", [
    (8, 640, 2048, "bf16", None), (3, 641, 2496, "bf16", None), (2, 700, 1284, "f32", None),
    (16, 41, 2560, "bf16", 8), (1, 37, 1024, "f32", 7), (5, 40, 2568, "bf16", 8),
    (4, 420, 2888, "bf16", None), (2, 2500, 4096, "bf16", None), (3, 14, 1900, "f32", 2),
    (2, 700, 4096, "bf16", None), (9, 330, 5000, "bf16", None), (2, 320, 12288, "bf16", None),
    (6, 7, 12296, "bf16", 1)])
def test_rows_through_the_ring(n_parts, T, H, dtype, max_sms, quant):
    """Rows around the sizes at which a ring's pipelines change, few and many to a CTA."""
    for in_place in (False, True):
        check(n_parts, T, H, dtype, gate_tokens=3 if T % 2 else None, max_sms=max_sms, quant=quant,
              in_place=in_place, t0=1, t1=T - 1, n_out=2, block_scale=0.5)


@pytest.mark.parametrize("quant", [None, "e4m3"])
@pytest.mark.parametrize("n_parts,T,H,dtype", [
    (3, 2600, 248, "bf16"), (8, 2500, 512, "bf16"), (2, 1300, 1016, "bf16"), (5, 700, 1992, "bf16"),
    (1, 2450, 100, "f32"), (9, 1300, 508, "f32"), (4, 620, 1020, "f32"),
    (3, 600, 4096, "bf16"), (2, 1100, 2048, "bf16"), (5, 450, 5120, "bf16"), (4, 308, 3068, "f32"),
    (1, 340, 6144, "bf16"), (2, 605, 1996, "f32")])
def test_short_rows_beside_each_other(n_parts, T, H, dtype, quant):
    check(n_parts, T, H, dtype, post=T % 4 != 0, gate_tokens=7, quant=quant, in_place=True,
          t0=2, t1=T - 1, residual_scale=0.5)


@pytest.mark.parametrize("quant", [None, "e4m3"])
@pytest.mark.parametrize("T,t0,t1", [(9, 4, 7), (9, 0, 1), (9, 8, 9), (500, 3, 499), (9, 5, 5)])
def test_ranges_and_in_place(T, t0, t1, quant):
    for in_place in (False, True):
        check(4, T, 1024, "bf16", gate_tokens=2, t0=t0, t1=t1, quant=quant, in_place=in_place,
              n_out=2)


@pytest.mark.parametrize("T", [2, 200])
def test_rows_without_a_block_or_a_residual(T):
    """Zero rows: the block's norm of a zero row is zero (eps keeps it finite), a row
    that is zero throughout gives zeros; scales of 0 leave one term."""
    for dtype in DTYPES:
        host, block = make(2, T, 1024, dtype, gate_tokens=1)
        for p in host["partials"]:
            p[0] = 0
        host["residual"][1] = 0
        block["gate"][1] = 0
        d, b = on_gpu(host, block)
        for bs, rs in ((1.0, 1.0), (0.0, 1.0), (1.0, 0.0), (0.0, 0.0)):
            out, res = [torch.empty_like(d["residual"])], torch.empty_like(d["residual"])
            tw.tw_fused_reduce_postnorm_add_rmsnorm(
                d["partials"], d["residual"], d["weight"], out, res, EPS, block_scale=bs,
                residual_scale=rs, **b)
            x, y, ex, ey = expected(host, block, eps=EPS, block_scale=bs, residual_scale=rs)
            close(res, x, ex, (dtype, bs, rs))
            close(out[0], y, ey, (dtype, bs, rs))
            assert not res[1].any() and not out[0][1].any()


@pytest.mark.parametrize("T", [3, 300])
def test_nan_and_infinities_stay_in_their_row(T):
    for dtype in DTYPES:
        host, block = make(3, T, 512, dtype)
        host["partials"][1][0, 5] = float("nan")
        host["residual"][1, 7] = float("inf")
        d, b = on_gpu(host, block)
        out, res = [torch.empty_like(d["residual"])], torch.empty_like(d["residual"])
        tw.tw_fused_reduce_postnorm_add_rmsnorm(d["partials"], d["residual"], d["weight"], out,
                                                res, EPS, **b)
        x, y, ex, ey = expected(host, block, eps=EPS)
        close(res[2:], x[2:], ex[2:], dtype)
        close(out[0][2:], y[2:], ey[2:], dtype)
        assert res[0].isnan().all() and out[0][0].isnan().all()
        assert res[1, 7] == float("inf") and out[0][1, 7].isnan()
        assert torch.all(out[0][1, torch.arange(512) != 7] == 0)
        q, qs = [torch.empty(T, 512, dtype=torch.int8, device="cuda")], [torch.empty(T, device="cuda")]
        tw.tw_fused_reduce_postnorm_add_rmsnorm_q8(d["partials"], d["residual"], d["weight"], q,
                                                   qs, res, EPS, **b)
        assert qs[0][:2].isnan().all() and not q[0][:2].any() and qs[0][2:].isfinite().all()


def test_nearly_cancelling_block_and_residual():
    """x is a small difference of large terms: its norm is taken from x itself."""
    host, block = make(1, 50, 2048, "f32")
    s = host["partials"][0].double()
    u = s / (s.square().mean(1, keepdim=True) + EPS).sqrt() * block["post_weight"].double()
    host["residual"] = (-u + 1e-3 * host["residual"].double()).float()
    d, b = on_gpu(host, block)
    out, res = [torch.empty_like(d["residual"])], torch.empty_like(d["residual"])
    tw.tw_fused_reduce_postnorm_add_rmsnorm(d["partials"], d["residual"], d["weight"], out, res,
                                            0.0, post_eps=EPS, **b)
    x, y, ex, ey = expected(host, block, eps=0.0, post_eps=EPS)
    close(res, x, ex, "x")
    close(out[0], y, ey, "y")


@pytest.mark.parametrize("T", [1, 60, 1000])
def test_without_norm_gate_and_scales_it_is_the_plain_step(T):
    wl = inputs.Workload("plain", 4, T, 2048, "bf16", EPS, 1, 8)
    d = inputs.make_inputs(wl, device="cuda")
    outs = []
    for call in (tw.tw_fused_reduce_add_rmsnorm, tw.tw_fused_reduce_postnorm_add_rmsnorm):
        out, res = [torch.empty_like(d["residual"])], torch.empty_like(d["residual"])
        call(d["partials"], d["residual"], d["weight"], out, res, EPS)
        outs.append((out[0], res))
    assert torch.equal(outs[0][1], outs[1][1])
    # The sums of squares may be taken in another order.
    diff = (outs[0][0].float() - outs[1][0].float()).abs()
    assert torch.all(diff <= 2.0 ** -7 * outs[0][0].float().abs())


@pytest.mark.parametrize("T", [4, 500])
def test_two_streams_and_a_replayed_graph(T):
    host, block = make(2, T, 4096, "bf16", gate_tokens=7)
    d, b = on_gpu(host, block)
    outs = [([torch.zeros_like(d["residual"])], torch.zeros_like(d["residual"])) for _ in range(4)]
    torch.cuda.synchronize()

    def run(out, res, stream=None):
        tw.tw_fused_reduce_postnorm_add_rmsnorm(d["partials"], d["residual"], d["weight"], out,
                                                res, EPS, gate_tokens=7, stream=stream, **b)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, o in enumerate(outs):
        run(*o, stream=streams[i % 2])
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o[0][0], outs[0][0][0]) and torch.equal(o[1], outs[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*outs[0])
        run(*outs[1])
    host, block = make(2, T, 4096, "bf16", gate_tokens=7, seed=5)
    d2, b2 = on_gpu(host, block)
    for p, q in zip(d["partials"] + [d["residual"], d["weight"], b["gate"], b["post_weight"]],
                    d2["partials"] + [d2["residual"], d2["weight"], b2["gate"], b2["post_weight"]]):
        p.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    x, y, ex, ey = expected(host, block, eps=EPS, gate_tokens=7)
    for out, res in outs[:2]:
        close(res, x, ex, "x")
        close(out[0], y, ey, "y")


def test_past_2_31_elements():
    T, H = 140000, 16384  # 2.3e9
    p = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    residual = torch.zeros_like(p)
    host, block = make(1, 5, H, "bf16", gate_tokens=1)
    p[-5:], residual[-5:] = host["partials"][0].cuda(), host["residual"].cuda()
    gate = torch.zeros_like(p)
    gate[-5:] = block["gate"].cuda()
    out, res = torch.empty_like(p), torch.empty_like(p)
    tw.tw_fused_reduce_postnorm_add_rmsnorm([p], residual, host["weight"].cuda(), [out], res, EPS,
                                            post_weight=block["post_weight"].cuda(), gate=gate)
    x, y, ex, ey = expected(host, block, eps=EPS)
    close(res[-5:], x, ex, "x")
    close(out[-5:], y, ey, "y")
    assert not res[:-5].any() and not out[:-5].any()
