"""The operators of a layer with sandwich norms and 4-bit weights in a row, as a decode
step calls them: every step against the formulas in 64 bits on what it was given."""
import numpy as np
import pytest
import torch

from reduce_residual_rmsnorm_tw_gb300 import layer_step, tw
from tests import w4_reference as ref
from tests.postnorm_reference import step
from tests.q8_reference import KIND, check_rows, f64

pytestmark = pytest.mark.gpu
EPS = 1e-5


class Layer:
    """Two linear layers (H -> H) in 4 bits with the norms behind each."""

    def __init__(self, T, H, parts, kinds, quant, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda")
        self.T, self.H, self.quant = T, H, quant
        self.w4, self.parts, self.norms = [], [], []
        for kind, group in kinds:
            q = tw.W4Weight(H, H, group, kind)
            tw.tw_quantize_w4((normal(H, H) / H ** 0.5).to(dtype), q)
            self.w4.append(q)
            self.parts.append([normal(T, H).to(dtype) for _ in range(parts)])
            self.norms.append({"weight": (normal(H).abs() + 0.5).to(dtype),
                               "post_weight": (normal(H).abs() + 0.5).to(dtype),
                               "gate": normal(1, H).to(dtype)})
        self.residual = [normal(T, H).to(dtype) for _ in range(3)]
        self.x = normal(T, H).to(dtype)
        self.q = [torch.zeros(T, H, dtype=KIND[quant], device="cuda") for _ in range(2)]
        self.scale = [torch.zeros(T, device="cuda") for _ in range(2)]

    def run(self, stream=None):
        """x -> layer 0 -> 8-bit rows -> layer 1 -> 8-bit rows."""
        for i in range(2):
            n = self.norms[i]
            layer_step.sandwich_layer_step_w4(
                self.x if i == 0 else self.q[0], self.w4[i], self.parts[i], self.residual[i],
                n["weight"], [self.q[i]], self.residual[i + 1], EPS,
                x_scale=None if i == 0 else self.scale[0], out_scale=[self.scale[i]],
                stream=stream, post_weight=n["post_weight"], gate=n["gate"],
                gate_tokens=self.T, block_scale=0.5)

    def check(self):
        for i in range(2):
            values, scales, _ = ref.unpack(self.w4[i])
            x = f64(self.x) if i == 0 else f64(self.q[0]) * f64(self.scale[0])[:, None]
            want = x @ ref.weights(values, scales, self.w4[i].group).T
            got = self.parts[i][0]
            bound = ref.product_bound(x, ref.weights(values, scales, self.w4[i].group), want,
                                      self.w4[i].group, got.dtype,
                                      i == 0 and self.x.dtype == torch.float32)
            assert np.all(np.abs(f64(got) - want) <= bound), f"product {i}"
            n = {k: f64(v) for k, v in self.norms[i].items()}
            d = {"partials": [f64(p) for p in self.parts[i]], "residual": f64(self.residual[i]),
                 "weight": n["weight"]}
            res, y, er, ey = step(d, n["post_weight"], n["gate"], self.T, 0.5, eps=EPS)
            r = f64(self.residual[i + 1])
            half = torch.finfo(self.residual[0].dtype).eps / 2
            assert np.all(np.abs(r - res) <= er + half * (np.abs(res) + er)), f"residual {i}"
            rel = ey.max(axis=1) / np.abs(y).max(axis=1) + 6 * 2.0 ** -24
            check_rows(self.q[i], self.scale[i], y, self.quant, rel, f"rows {i}")


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("T,H,parts", [(1, 2048, 2), (7, 1024, 3), (20, 4096, 1)])
def test_two_layers(T, H, parts, quant):
    layer = Layer(T, H, parts, [("int4", 128), ("e2m1", 32)], quant)
    layer.run()
    torch.cuda.synchronize()
    layer.check()
    assert tw.tw_device_status() == 0


def test_fp32_layers_on_a_stream_of_their_own():
    layer = Layer(3, 1024, 2, [("e2m1", 64), ("int4", 32)], "int8", torch.float32)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    layer.run(stream)
    stream.synchronize()
    layer.check()


@pytest.mark.parametrize("T", [1, 9])
def test_a_captured_step_replayed_on_new_inputs(T):
    layer = Layer(T, 2048, 2, [("int4", 64), ("int4", 128)], "int8")
    layer.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run()
    g = torch.Generator(device="cuda").manual_seed(99)
    for t in (layer.x, layer.residual[0], layer.parts[0][1], layer.parts[1][1]):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    for t in layer.q + layer.scale:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    layer.check()


def test_two_layers_at_once_on_two_streams():
    a = Layer(5, 2048, 2, [("int4", 128), ("int4", 128)], "int8", seed=1)
    b = Layer(11, 2048, 1, [("e2m1", 32), ("int4", 64)], "e4m3", seed=2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):  # residual 0 is only read, so every run gives the same
        a.run(streams[0])
        b.run(streams[1])
    torch.cuda.synchronize()
    a.check()
    b.check()


@pytest.mark.parametrize("T", [32, 33, 130])
def test_many_tokens_by_the_weights_read_back(T):
    """With a workspace, from w4_library_tokens on: the product of the bf16 weights that
    tw_dequantize_w4 gives (their rounding, half a bf16 step each, is in the bound)."""
    H, K = 512, 1024
    g = torch.Generator(device="cuda").manual_seed(T)
    w = torch.randn(H, K, generator=g, device="cuda") / K ** 0.5
    w4 = tw.W4Weight(H, K, 64, "int4")
    tw.tw_quantize_w4(w, w4)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    partials = [torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2)]
    other = partials[1].clone()
    residual = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    weight = torch.rand(H, generator=g, device="cuda").bfloat16()
    out, res = [torch.empty_like(residual)], torch.empty_like(residual)
    workspace = torch.full((H, K), 7.0, dtype=torch.bfloat16, device="cuda")
    layer_step.sandwich_layer_step_w4(x, w4, partials, residual, weight, out, res, EPS,
                                      workspace=workspace, post_weight=weight)
    torch.cuda.synchronize()
    values, scales, _ = ref.unpack(w4)
    w64 = ref.weights(values, scales, 64)
    library = T >= layer_step.w4_library_tokens(H, K)
    assert bool(torch.all(workspace == 7)) != library
    if library:
        w64 = f64(torch.from_numpy(w64).to(torch.bfloat16))
        assert np.array_equal(f64(workspace), w64)
    want = f64(x) @ w64.T
    # A library sum of K terms in fp32, in any order, rounded to bf16.
    bound = 2.0 ** -8 * np.abs(want) + K * 2.0 ** -23 * (np.abs(f64(x)) @ np.abs(w64).T)
    assert np.all(np.abs(f64(partials[0]) - want) <= bound)
    assert torch.equal(partials[1], other)
    d = {"partials": [f64(p) for p in partials], "residual": f64(residual), "weight": f64(weight)}
    r64, y, er, ey = step(d, f64(weight), eps=EPS)
    for got, ref64, err in ((res, r64, er), (out[0], y, ey)):
        assert np.all(np.abs(f64(got) - ref64) <= err + 2.0 ** -8 * (np.abs(ref64) + err))


def test_other_streams_of_other_calls_see_whole_results():
    """The weights are laid out on one stream and used on another behind an event."""
    H = 1024
    w = torch.randn(H, H, device="cuda").bfloat16()
    w4 = tw.W4Weight(H, H, 128, "e2m1")
    x = torch.randn(4, H, device="cuda").bfloat16()
    outs = [torch.empty(4, H, device="cuda") for _ in range(2)]
    tw.tw_quantize_w4(w, w4)
    tw.tw_gemm_w4(x, w4, outs[0])
    torch.cuda.synchronize()
    w4.packed.zero_()
    s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    tw.tw_quantize_w4(w, w4, stream=s0)
    event = torch.cuda.Event()
    event.record(s0)
    s1.wait_event(event)
    tw.tw_gemm_w4(x, w4, outs[1], stream=s1)
    s1.synchronize()
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("T,H", [(1, 512), (6, 2048), (24, 4096)])
def test_weights_laid_out_again_just_before_they_are_used(T, H):
    """Calls right behind each other see what the one before wrote, not what was there."""
    g = torch.Generator(device="cuda").manual_seed(H)
    ws = [torch.randn(H, H, generator=g, device="cuda").bfloat16() for _ in range(6)]
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w4 = tw.W4Weight(H, H, 64, "int4")
    apart = [[torch.zeros(T, H, device="cuda"), torch.zeros_like(ws[0])] for _ in ws]
    for w, (out, back) in zip(ws, apart):
        for call in (lambda: tw.tw_quantize_w4(w, w4), lambda: tw.tw_gemm_w4(x, w4, out),
                     lambda: tw.tw_dequantize_w4(w4, back)):
            call()
            torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    got = [[torch.zeros_like(out), torch.zeros_like(back)] for out, back in apart]
    with torch.cuda.graph(graph):
        for w, (out, back) in zip(ws, got):
            tw.tw_quantize_w4(w, w4)
            tw.tw_gemm_w4(x, w4, out)
            tw.tw_dequantize_w4(w4, back)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for (a, b), (c, d) in zip(apart, got):
        assert torch.equal(a, c) and torch.equal(b, d)


def test_two_graphs_replayed_at_once():
    """Captured calls share nothing: two graphs of one layer's weights beside each other."""
    layers = [Layer(9, 2048, 2, [("int4", 128), ("e2m1", 64)], "int8", seed=3) for _ in range(2)]
    layers[1].w4 = layers[0].w4
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for layer in layers:
        layer.run()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(4):
                layer.run()
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for layer in layers:
        layer.check()
    assert tw.tw_device_status() == 0
