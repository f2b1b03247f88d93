"""The 8-bit operators together, as a layer uses them: the norm's 8-bit rows
through a product, its output quantised and multiplied into a partial, and the
next norm on that partial.  Nothing waits between the calls; every stage is
then compared with the 64-bit reference of that stage on the stage's actual
inputs."""
import numpy as np
import pytest
import torch

import oracle
from reduce_residual_rmsnorm_tw_gb300 import inputs, layer_step, tw
from reduce_residual_rmsnorm_tw_gb300.inputs import Workload
from tests.parity import check_close
from tests.q8_reference import KIND, U, check_product, check_rows, draw_8_bit, row_error

pytestmark = pytest.mark.gpu


def check_norm_stage(wl, parts, res, weight, q, s, res_out, quant, what):
    p64 = [inputs.to_f64(p) for p in parts]
    r64, w64 = inputs.to_f64(res), inputs.to_f64(weight)
    ref, ref_res = oracle.reordered(p64, r64, w64, wl.eps, n_out=1)
    rel = 2 * row_error([p * w64 for p in p64 + [r64]], (sum(p64) + r64) * w64) + 100 * U
    check_rows(q, s, ref[0], quant, rel, what)
    check_close(res_out, ref_res, wl.dtype, what)


class Chain:
    """norm -> up -> quantise -> down into partial 1 -> norm, buffers and all."""

    def __init__(self, T, H, K, quant, seed):
        self.wl = Workload(f"chain_{T}", 3, T, H, "bf16", 1e-5, 1, seed, partial_std=0.5)
        self.quant, self.T, self.H, self.K = quant, T, H, K
        d = inputs.make_inputs(self.wl, device="cuda")
        self.parts, self.res, self.weight = d["partials"], d["residual"], d["weight"]
        self.up, self.up_s = draw_8_bit(K, H, quant, seed + 1)
        self.down, self.down_s = draw_8_bit(H, K, quant, seed + 2)
        self.up_s *= 0.01
        self.down_s *= 0.01

        def rows(n, kind):
            return torch.empty(T, n, dtype=kind, device="cuda")
        kind, bf = KIND[quant], torch.bfloat16
        self.q = [rows(H, kind), rows(K, kind), rows(H, kind)]
        self.s = [torch.empty(T, device="cuda") for _ in range(3)]
        self.mid, self.down_out = rows(K, bf), rows(H, bf)
        self.res1, self.res2 = rows(H, bf), rows(H, bf)

    def run(self):
        tw.tw_fused_reduce_add_rmsnorm_q8(self.parts, self.res, self.weight, self.q[:1],
                                          self.s[:1], self.res1, self.wl.eps)
        tw.tw_gemm_q8(self.q[0], self.s[0], self.up, self.up_s, self.mid)
        tw.tw_quantize_rows_q8(self.mid, self.q[1], self.s[1])
        tw.tw_gemm_q8(self.q[1], self.s[1], self.down, self.down_s, self.down_out)
        tw.tw_fused_reduce_add_rmsnorm_q8([self.parts[0], self.down_out], self.res1, self.weight,
                                          self.q[2:], self.s[2:], self.res2, self.wl.eps)

    def check(self):
        check_norm_stage(self.wl, self.parts, self.res, self.weight, self.q[0], self.s[0],
                         self.res1, self.quant, "first norm")
        check_product(self.mid, self.q[0], self.s[0], self.up, self.up_s, "up")
        check_rows(self.q[1], self.s[1], inputs.to_f64(self.mid), self.quant,
                   np.full(self.T, 3 * U), "quantised")
        check_product(self.down_out, self.q[1], self.s[1], self.down, self.down_s, "down")
        check_norm_stage(self.wl, [self.parts[0], self.down_out], self.res1, self.weight,
                         self.q[2], self.s[2], self.res2, self.quant, "second norm")

    def outputs(self):
        return [t.view(torch.uint8) for t in self.q] + self.s + [self.mid, self.down_out,
                                                                 self.res1, self.res2]


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("T", [1, 6, 70, 500])
def test_layer_chain(T, quant):
    c = Chain(T, 1024, 2000, quant, 91)
    c.run()
    torch.cuda.synchronize()
    c.check()
    assert tw.tw_device_status() == 0


@pytest.mark.parametrize("T", [2, 200])
def test_captured_chain_replays_on_new_inputs(T):
    a, b = Chain(T, 1024, 2000, "int8", 92), Chain(T, 1024, 2000, "int8", 95)
    a.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
    # Replay on b's inputs, beside b's own eager chain on another stream.
    for mine, theirs in zip(a.parts + [a.res, a.weight, a.up, a.up_s, a.down, a.down_s],
                            b.parts + [b.res, b.weight, b.up, b.up_s, b.down, b.down_s]):
        mine.view(torch.uint8).copy_(theirs.view(torch.uint8))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g.replay()
    with torch.cuda.stream(side):
        b.run()
    torch.cuda.synchronize()
    a.check()
    for x, y in zip(a.outputs(), b.outputs()):
        assert torch.equal(x, y)


def test_two_graphs_at_once():
    # Two captured chains replayed on two streams share no state.
    a, b = Chain(40, 1024, 2000, "e4m3", 96), Chain(300, 1024, 2000, "int8", 97)
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for c in (a, b):
        c.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for c in (a, b):
        for t in c.outputs():
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    a.check()
    b.check()
    assert tw.tw_device_status() == 0


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("T,split", [(600, None), (70, 3)])
def test_two_chunk_layer_step_q8(T, split, quant):
    wl = Workload(f"step_q8_{T}", 4, T, 2048, "bf16", 1e-5, 1, 98, partial_std=0.5)
    d = inputs.make_inputs(wl, device="cuda")
    x, xs = draw_8_bit(T, 1536, quant, 99)
    w, ws = draw_8_bit(2048, 1536, quant, 100)
    ws *= 0.01
    q = [torch.empty(T, 2048, dtype=KIND[quant], device="cuda")]
    s = [torch.empty(T, device="cuda")]
    res_out = torch.empty_like(d["residual"])
    g, f = torch.cuda.Stream(), torch.cuda.Stream(priority=-1)
    for st in (g, f):
        st.wait_stream(torch.cuda.current_stream())
    layer_step.two_chunk_layer_step_q8(x, xs, w, ws, d["partials"], d["residual"], d["weight"],
                                       q, s, res_out, wl.eps, 16, g, f, t_split=split)
    torch.cuda.current_stream().wait_stream(g)
    torch.cuda.synchronize()
    check_product(d["partials"][0], x, xs, w, ws, "partial 0")
    check_norm_stage(wl, d["partials"], d["residual"], d["weight"], q[0], s[0], res_out, quant,
                     "step")
    assert tw.tw_device_status() == 0
