"""One mixture-of-experts layer of a mixed-precision decoder, between its attention and the next layer's: 8-bit output
projection, residual and RMS norm in one pass, router, 4-bit experts, the next norm and an 8-bit head, as one captured
graph a step. With --context the layer's attention too: 8-bit query, key and value projection, rotation and append to a paged
8-bit cache, attention of each sequence's new token. Random weights.

    python examples/mixed_layer.py [--tokens T] [--width D] [--inner I] [--experts E] [--topk k] [--outputs N] [--steps S]
                                   [--context C] [--kv-heads H]

Prints the time of a step and the rate at which it reads the weights that its tokens use.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import microscaling_fp4_quantized_amd as F  # noqa: E402


class Attention:
    """The attention of T sequences in front of the layer: its projection, the cache, and the buffers of a step. A sequence holds up to
    `most` tokens in pages of `page`."""

    def __init__(self, T, D, most, kv_heads=2, dim=64, page=32, window=0, sinks=0, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed + 1)
        if D % (dim * kv_heads):
            raise ValueError(f"the width {D} must be a multiple of {kv_heads} key-value heads of {dim}")
        self.Hq, self.H, self.dim, self.window, self.sinks = D // dim, kv_heads, dim, window, sinks
        f8, f32, bf = torch.float8_e4m3fn, torch.float32, torch.bfloat16
        rows = (self.Hq + 2 * kv_heads) * dim
        self.proj = F.fp8_quantize_weights((torch.randn(rows, D, generator=gen, device=device) * D ** -0.5).to(bf))
        cols = -(-most // page)
        # pages of a pool in any order; unused places of a page may hold anything
        self.table = torch.randperm(T * cols, generator=gen, device=device).to(torch.int32).view(T, cols)
        self.lengths = torch.zeros(T, dtype=torch.int32, device=device)
        self.pages = [torch.empty(T * cols, kv_heads, page, dim, dtype=f8, device=device) for _ in range(2)]
        self.scales = dict(zip(("k_scales", "v_scales"), (torch.empty(T * cols, kv_heads, page, device=device) for _ in range(2))))
        self.freqs = (1e4 ** (-torch.arange(dim // 2, dtype=torch.float64, device=device) * 2 / dim)).to(f32)
        self.x = torch.randn(T, D, generator=gen, device=device).to(bf)  # the layer's normed input
        self.x8 = torch.empty(T, D, dtype=f8, device=device), torch.empty(T, D // 128, dtype=f32, device=device)
        self.qkv = torch.empty(T, rows, dtype=bf, device=device)
        self.q = torch.empty(T, self.Hq, dim, dtype=bf, device=device)
        self.ws = torch.empty(F.attention_workspace_bytes(T, T, self.Hq, kv_heads, dim), dtype=torch.uint8, device=device)

    def cache(self):
        return *self.pages, self.table, self.lengths

    def prompt(self, x):
        """C more tokens of each sequence, x [T, C, D]: what they attend to, [T * C, D]."""
        T, C, D = x.shape
        flat = x.reshape(T * C, D)
        q, k, v = self._heads(F.fp8_linear(*F.fp8_quantize(flat), *self.proj))
        self.lengths += C
        starts = torch.arange(0, T * C + 1, C, dtype=torch.int32, device=x.device)
        q = F.fp4_kv_append(k, v, *self.cache(), starts, q=q, freqs=self.freqs, **self.scales)
        return F.fp4_attention_prompt(q, *self.cache(), starts, window=self.window, sinks=self.sinks, **self.scales).view(T * C, D)

    def step(self, out):
        """One token more of each sequence: attention of x's tokens into out [T, D]."""
        F.fp8_quantize(self.x, out=self.x8)
        q, k, v = self._heads(F.fp8_linear(*self.x8, *self.proj, out=self.qkv))
        self.lengths += 1
        F.fp4_kv_append(k, v, *self.cache(), q=q, freqs=self.freqs, out=self.q, **self.scales)
        F.fp4_attention_decode(self.q, *self.cache(), window=self.window, sinks=self.sinks, out=out.view(-1, self.Hq, self.dim),
                               workspace=self.ws, **self.scales)

    def _heads(self, qkv):
        qkv = qkv.view(-1, self.Hq + 2 * self.H, self.dim)
        return qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.H], qkv[:, self.Hq + self.H:]


class MixedLayer:
    """The layer's quantized weights, and the buffers of a step of T tokens; `attention` in front of it, or what it gave in attn."""

    def __init__(self, T, D, I, E, k, N, block=32, seed=0, device="cuda", attention=None):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=gen, device=device) * scale).bfloat16()

        def new(dtype, *shape):
            return torch.empty(shape, dtype=dtype, device=device)

        f8, f32, bf = torch.float8_e4m3fn, torch.float32, torch.bfloat16
        self.k, self.block, self.attention = k, block, attention
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
        if self.attention is not None:
            self.attention.step(self.attn)
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
        eight = [self.proj, self.head] + ([self.attention.proj] if self.attention is not None else [])
        return experts + self.router.numel() * 2 + sum(c.numel() + 4 * s.numel() for c, s in eight)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 1), ("width", 2048), ("inner", 768), ("experts", 128), ("topk", 8), ("outputs", 4096),
                        ("steps", 100), ("context", 0), ("kv-heads", 4)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    attention = None
    if a.context:
        attention = Attention(a.tokens, a.width, a.context + a.steps + 12, a.kv_heads, dim=128)
        for first in range(0, a.context, 512):  # the context in slices, as long prompts are served
            n = min(512, a.context - first)
            attention.prompt(torch.randn(a.tokens, n, a.width, device="cuda").bfloat16())
    layer = MixedLayer(a.tokens, a.width, a.inner, a.experts, a.topk, a.outputs, attention=attention)
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
    seen = f" over a context of {a.context}" if a.context else ""
    print(f"{a.tokens} token(s){seen}, width {a.width}, {a.topk} of {a.experts} experts of {a.inner}: {us:.1f} us a step, "
          f"{layer.weight_bytes() / us / 1e6:.2f} TB/s of weights")


if __name__ == "__main__":
    main()
