"""One mixture-of-experts layer of a mixed-precision decoder, between its attention and the next layer's: 8-bit output
projection, residual and RMS norm in one pass, router, 4-bit experts, the next norm and an 8-bit head, as one captured
graph a step. Random weights.

    python examples/mixed_layer.py [--tokens T] [--width D] [--inner I] [--experts E] [--topk k] [--outputs N] [--steps S]

Prints the time of a step and the rate at which it reads the weights that its tokens use.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import microscaling_fp4_quantized_amd as F  # noqa: E402


class MixedLayer:
    """The layer's quantized weights, and the buffers of a step of T tokens."""

    def __init__(self, T, D, I, E, k, N, block=32, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=gen, device=device) * scale).bfloat16()

        def new(dtype, *shape):
            return torch.empty(shape, dtype=dtype, device=device)

        f8, f32, bf = torch.float8_e4m3fn, torch.float32, torch.bfloat16
        self.k, self.block = k, block
        # quantized once, as a user's program would when it loads a model
        self.proj = F.fp8_quantize_weights(normal(D, D, scale=D ** -0.5))
        self.head = F.fp8_quantize_weights(normal(N, D, scale=D ** -0.5))
        self.norm1, self.norm2 = normal(D, scale=0.1) + 1, normal(D, scale=0.1) + 1
        self.router = normal(E, D, scale=D ** -0.5)
        w13 = F.fp4_quantize_weights(normal(E * 2 * I, D, scale=D ** -0.5), block)
        w2 = F.fp4_quantize_weights(normal(E * D, I, scale=I ** -0.5), block)
        self.experts = (w13[0].view(E, 2 * I, D // 2), w13[1].view(E, 2 * I, D // 32), w2[0].view(E, D, I // 2),
                        w2[1].view(E, D, I // 32))
        # the step's inputs and outputs
        self.attn, self.hidden = normal(T, D, scale=1), normal(T, D, scale=1)
        self.attn8 = new(f8, T, D), new(f32, T, D // 128)
        self.o = new(bf, T, D)
        self.n1 = new(f8, T, D), new(f32, T, D // 128), new(bf, T, D), new(bf, T, D)
        self.routed = new(torch.int32, T, k), new(f32, T, k)
        self.moe = new(bf, T, D)
        self.n2 = new(f8, T, D), new(f32, T, D // 128), new(bf, T, D), None
        self.y = new(bf, T, N)
        self.route_ws = new(torch.uint8, 16 * T * E)
        self.moe_ws = new(torch.uint8, F.moe_workspace_bytes(T, k, D, I))

    def step(self):
        """y = head(norm2(h + experts(norm1(h)))), h = hidden + proj(attn); self.n2[2] is the next layer's residual."""
        F.fp8_quantize(self.attn, out=self.attn8)
        F.fp8_linear(*self.attn8, *self.proj, out=self.o)
        _, _, h, n = F.fp8_add_rmsnorm_quantize(self.o, self.norm1, self.hidden, normed=True, out=self.n1)
        F.fp4_moe_route(n, self.router, self.k, out=self.routed, workspace=self.route_ws)
        F.fp4_moe_experts(n, *self.routed, *self.experts, self.block, out=self.moe, workspace=self.moe_ws)
        codes, scales, _, _ = F.fp8_add_rmsnorm_quantize(self.moe, self.norm2, h, out=self.n2)
        return F.fp8_linear(codes, scales, *self.head, out=self.y)

    def capture(self):
        """The step as a graph: replay() runs it on the inputs that attn and hidden hold then."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()  # first-use setup happens outside the capture
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph

    def weight_bytes(self):
        """Bytes of the weights that the last step's tokens use."""
        E = self.router.shape[0]
        used = self.routed[0].unique().numel()
        experts = sum(t.numel() for t in self.experts) * used // E
        return experts + self.router.numel() * 2 + sum(c.numel() + 4 * s.numel() for c, s in (self.proj, self.head))


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 1), ("width", 2048), ("inner", 768), ("experts", 128), ("topk", 8), ("outputs", 4096),
                        ("steps", 100)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    layer = MixedLayer(a.tokens, a.width, a.inner, a.experts, a.topk, a.outputs)
    graph = layer.capture()
    for _ in range(10):
        graph.replay()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(end) * 1e3 / a.steps
    print(f"{a.tokens} token(s), width {a.width}, {a.topk} of {a.experts} experts of {a.inner}: {us:.1f} us a step, "
          f"{layer.weight_bytes() / us / 1e6:.2f} TB/s of weights")


if __name__ == "__main__":
    main()
