"""How the 8-bit and mixture-of-experts operators are called: the compiled argument checks and binding.py's own give the
same bits and refuse the same operands, side streams and replayed graphs give the results of one call after another.

(The results themselves are checked against float64 by the operators' own tests.)
"""
import pytest
import torch

import microscaling_fp4_quantized_amd as F
from microscaling_fp4_quantized_amd import binding as B
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


def normal(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


class Layer:
    """Weights, inputs and given outputs of one call of every operator; T tokens of D, strided by 8 more."""

    def __init__(self, seed, T, D=512, I=256, E=8, k=3, N=300, block=32):
        self.T, self.D, self.k, self.block = T, D, k, block
        self.x = normal(seed, T, D + 8)[:, :D]
        self.r = normal(seed + 1, T, D + 16)[:, :D]
        self.g = normal(seed + 2, D)
        self.wr = normal(seed + 3, E, D, scale=D ** -0.5)
        self.w = normal(seed + 4, N, D, scale=D ** -0.5)
        w13 = F.fp4_quantize_weights(normal(seed + 5, E * 2 * I, D, scale=D ** -0.5), block)
        w2 = F.fp4_quantize_weights(normal(seed + 6, E * D, I, scale=I ** -0.5), block)
        self.experts = (w13[0].view(E, 2 * I, D // 2), w13[1].view(E, 2 * I, D // 32), w2[0].view(E, D, I // 2),
                        w2[1].view(E, D, I // 32))

        def new(dtype, *shape):
            return torch.empty(shape, dtype=dtype, device=DEV)
        f8, f32, bf = torch.float8_e4m3fn, torch.float32, torch.bfloat16
        self.norm_out = (new(f8, T, D), new(f32, T, D // 128), new(bf, T, D), new(bf, T, D))
        self.x_out = (new(f8, T, D), new(f32, T, D // 128))
        self.w_out = (new(f8, N, D), new(f32, -(-N // 128), D // 128))
        self.y = new(bf, T, N)
        self.route_out = (new(torch.int32, T, k), new(f32, T, k))
        self.route_ws = new(torch.uint8, 16 * T * E)
        self.moe = new(bf, T, D)
        self.moe_ws = new(torch.uint8, F.moe_workspace_bytes(T, k, D, I))

    def run(self, x=None):
        x = self.x if x is None else x
        F.fp8_quantize(x, out=self.x_out)
        F.fp8_quantize_weights(self.w, out=self.w_out)
        F.fp8_add_rmsnorm_quantize(x, self.g, self.r, normed=True, out=self.norm_out)
        F.fp8_linear(*self.norm_out[:2], *self.w_out, out=self.y)
        F.fp4_moe_route(self.norm_out[3], self.wr, self.k, out=self.route_out, workspace=self.route_ws)
        F.fp4_moe_experts(self.norm_out[3], *self.route_out, *self.experts, self.block, out=self.moe,
                          workspace=self.moe_ws)

    def outputs(self):
        return [*self.x_out, *self.w_out, *self.norm_out, self.y, *self.route_out, self.moe]

    def copies(self):
        return [bits(t).clone() for t in self.outputs()]

    def clear(self):
        for t in self.outputs():
            bits(t).fill_(0x55)


def bits(t):
    return t.view(torch.uint8)


def same(layer, want):
    return [i for i, (t, w) in enumerate(zip(layer.outputs(), want)) if not torch.equal(bits(t), w)]


SIZES = [1, 7, 40, 128]  # the experts of 128 tokens go through the pairs sorted by expert, of fewer straight to the pairs


def test_the_compiled_checks_are_built_and_used():
    assert B._fast(torch.empty(1, device=DEV)) is not None


@pytest.mark.parametrize("T", SIZES)
def test_compiled_and_python_checks_give_the_same_bits(T, monkeypatch):
    say(f"calls T {T}")
    layer = Layer(T, T)
    layer.run()
    torch.cuda.synchronize()
    want = layer.copies()
    monkeypatch.setattr(B, "_FAST", False)
    layer.clear()
    layer.run()
    torch.cuda.synchronize()
    assert not same(layer, want)
    # and with outputs and workspaces of the calls' own
    c, s, h, n = F.fp8_add_rmsnorm_quantize(layer.x, layer.g, layer.r, normed=True)
    wc, ws = F.fp8_quantize_weights(layer.w)
    ids, p = F.fp4_moe_route(n, layer.wr, layer.k)
    own = [*F.fp8_quantize(layer.x), wc, ws, c, s, h, n, F.fp8_linear(c, s, wc, ws), ids, p,
           F.fp4_moe_experts(n, ids, p, *layer.experts, layer.block)]
    assert all(torch.equal(bits(a), w) for a, w in zip(own, want))


@pytest.mark.parametrize("compiled", [True, False])
def test_wrong_operands_are_refused(compiled, monkeypatch):
    """Nothing is launched for them: outputs keep what they held."""
    if not compiled:
        monkeypatch.setattr(B, "_FAST", False)
    a, b = Layer(1, 4), Layer(2, 5)
    host = a.x.cpu()
    a.run()
    torch.cuda.synchronize()
    want = a.copies()
    no, ro = a.norm_out, a.route_out
    codes, scales, wq, ws = *no[:2], *a.w_out
    nn, ex = no[3], a.experts
    bad = [
        lambda: F.fp8_quantize(a.x, out=b.x_out),
        lambda: F.fp8_quantize(a.x.float(), out=a.x_out),
        lambda: F.fp8_quantize(a.x[0], out=a.x_out),
        lambda: F.fp8_quantize(a.x, out=(a.x_out[0].view(torch.uint8), a.x_out[1])),
        lambda: F.fp8_quantize(a.x, out=(a.x_out[0], a.x_out[1].double())),
        lambda: F.fp8_quantize(normal(9, 512, 4).t(), out=a.x_out),
        lambda: F.fp8_quantize_weights(a.w, out=(a.w_out[0], a.w_out[1][:1])),
        lambda: F.fp8_add_rmsnorm_quantize(a.x, a.g[:256], a.r, normed=True, out=no),
        lambda: F.fp8_add_rmsnorm_quantize(a.x, a.g, b.r, normed=True, out=no),
        lambda: F.fp8_add_rmsnorm_quantize(a.x, a.g, None, normed=True, out=no),
        lambda: F.fp8_add_rmsnorm_quantize(a.x, a.g, a.r, normed=False, out=no),
        lambda: F.fp8_add_rmsnorm_quantize(a.x, a.g, a.r, normed=True, out=(*no[:3], b.norm_out[3])),
        lambda: F.fp8_linear(codes, scales, wq, ws, out=b.y),
        lambda: F.fp8_linear(codes, scales[:, :2], wq, ws, out=a.y),
        lambda: F.fp8_linear(codes, scales.t().contiguous().t(), wq, ws, out=a.y),
        lambda: F.fp8_linear(codes[:, :256], scales, wq, ws, out=a.y),
        lambda: F.fp8_linear(codes, scales, wq, ws[:2], out=a.y),
        lambda: F.fp8_linear(codes, scales, wq, ws, out=a.y.float()),
        lambda: F.fp8_linear(codes, scales, wq.cpu(), ws, out=a.y),
        lambda: F.fp4_moe_route(nn, a.wr[:, :256], a.k, out=ro, workspace=a.route_ws),
        lambda: F.fp4_moe_route(nn, a.wr, a.k, out=b.route_out, workspace=a.route_ws),
        lambda: F.fp4_moe_route(nn, a.wr, a.k + 1, out=ro, workspace=a.route_ws),
        lambda: F.fp4_moe_route(nn, a.wr, a.k, out=ro, workspace=a.route_ws[:-1]),
        lambda: F.fp4_moe_route(nn, a.wr, a.k, out=ro, workspace=None),
        lambda: F.fp4_moe_route(nn[0], a.wr, a.k, out=ro, workspace=a.route_ws),
        lambda: F.fp4_moe_route(nn, a.wr, a.k, out=(ro[0].long(), ro[1]), workspace=a.route_ws),
        lambda: F.fp4_moe_route(host, a.wr, a.k, out=ro, workspace=a.route_ws),
        lambda: F.fp4_moe_experts(nn, b.route_out[0], ro[1], *ex, 32, out=a.moe, workspace=a.moe_ws),
        lambda: F.fp4_moe_experts(nn, ro[0].long(), ro[1], *ex, 32, out=a.moe, workspace=a.moe_ws),
        lambda: F.fp4_moe_experts(nn, *ro, ex[0][:, :256], *ex[1:], 32, out=a.moe, workspace=a.moe_ws),
        lambda: F.fp4_moe_experts(nn, *ro, ex[0], ex[1][:4], *ex[2:], 32, out=a.moe, workspace=a.moe_ws),
        lambda: F.fp4_moe_experts(nn, *ro, ex[0], ex[1], ex[2][:4], ex[3], 32, out=a.moe, workspace=a.moe_ws),
        lambda: F.fp4_moe_experts(nn, *ro, *ex, 32, out=b.moe, workspace=a.moe_ws),
        lambda: F.fp4_moe_experts(nn, *ro, *ex, 32, out=a.moe, workspace=a.moe_ws[:-1]),
        lambda: F.fp4_moe_experts(nn, *ro, *ex, 32, out=a.moe, workspace=None),
        lambda: F.fp4_moe_experts(host, *ro, *ex, 32, out=a.moe, workspace=a.moe_ws),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    refused = [
        lambda: F.fp8_add_rmsnorm_quantize(a.x, a.g, a.r, eps=-1.0, normed=True, out=no),
        lambda: F.fp4_moe_experts(nn, *ro, *ex, 48, out=a.moe, workspace=a.moe_ws),
        lambda: F.fp8_quantize(a.x[:0], out=(a.x_out[0][:0], a.x_out[1][:0])),
        lambda: F.fp8_quantize(normal(3, 4, 517)[:, 5:], out=a.x_out),  # 10 bytes past a 16-byte boundary
    ]
    for call in refused:
        with pytest.raises(F.Fp4Error):
            call()
    torch.cuda.synchronize()
    assert not same(a, want)


@pytest.mark.parametrize("T", SIZES)
def test_side_streams_match_serial(T):
    say(f"operators on two streams, T {T}")
    layers = [Layer(10 * T + i, T) for i in range(4)]
    for layer in layers:
        layer.run()
    torch.cuda.synchronize()
    want = [layer.copies() for layer in layers]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for layer in layers:
            layer.clear()
        torch.cuda.synchronize()
        for i, layer in enumerate(layers):
            with torch.cuda.stream(streams[i % 2]):
                layer.run()
        torch.cuda.synchronize()
        assert [same(layer, w) for layer, w in zip(layers, want)] == [[]] * 4


@pytest.mark.parametrize("T", SIZES)
def test_graph_replays_match_eager(T):
    say(f"operators in a graph, T {T}")
    layer, other = Layer(T, T), normal(77, T, 512, scale=3.0)
    layer.run()
    torch.cuda.synchronize()
    want = layer.copies()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.run()
    for rep in range(5):
        layer.run(other)  # eager work on the same buffers between the replays
        torch.cuda.synchronize()
        assert same(layer, want)
        g.replay()
        torch.cuda.synchronize()
        assert not same(layer, want), rep
