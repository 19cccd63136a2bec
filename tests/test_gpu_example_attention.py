"""The attention in front of the example's layer: each of its stages against float64 on that stage's own inputs, and the step with it as a
graph against the eager one.

Bounds as in test_gpu_example.py: 2^-8 of a result in norm for the 8-bit product; the attention by paged_plain's own tolerance.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import fp8_plain
import paged_plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixed_layer.py")
    spec = importlib.util.spec_from_file_location("mixed_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


class Held:
    """What an attention's cache holds, in float64, as paged_plain.attention takes it."""

    def __init__(self, a):
        self.H, self.S, self.lengths = a.H, a.pages[0].shape[2], a.lengths.cpu()
        both = [p.float().cpu().double() * s.cpu().double()[..., None] for p, s in zip(a.pages, a.scales.values())]
        self.keys, self.values = ([pages[row[torch.arange(n) // self.S], :, torch.arange(n) % self.S]
                                   for row, n in zip(a.table.cpu().long(), self.lengths.tolist())] for pages in both)


@pytest.mark.parametrize("T,D,window,sinks", [(1, 256, 0, 0), (5, 384, 30, 2)])
def test_attention(example, T, D, window, sinks):
    a = example.Attention(T, D, 200, kv_heads=3 if D == 384 else 2, window=window, sinks=sinks)
    layer = example.MixedLayer(T, D, 128, 8, 2, 256, attention=a)
    g = torch.Generator("cuda").manual_seed(3)
    for C in (70, 41):
        got = a.prompt(torch.randn(T, C, D, generator=g, device="cuda").bfloat16())
        assert got.shape == (T * C, D) and got.isfinite().all()
    assert a.lengths.tolist() == [111] * T
    layer.step()
    torch.cuda.synchronize()
    assert a.lengths.tolist() == [112] * T
    qkv = fp8_plain.values(*a.x8, 1) @ fp8_plain.values(*a.proj, 128).T
    assert np.linalg.norm(a.qkv.cpu().double().numpy() - qkv) <= 2.0 ** -8 * np.linalg.norm(qkv)
    # the queries are rotated by the new token's place, and the cache's last entry by the same
    angle = 111.0 * a.freqs.cpu().double()[None].expand(T, -1)
    rows = a.qkv.cpu().double().view(T, -1, a.dim)
    want, tol = paged_plain.rotate(rows[:, :a.Hq], angle, False)
    assert ((a.q.cpu().double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()
    held = Held(a)
    want, tol = paged_plain.rotate(rows[:, a.Hq:a.Hq + a.H], angle, False)
    last = torch.stack([k[-1] for k in held.keys])
    top = want.abs().amax(-1, keepdim=True)
    assert ((last - want).abs() <= 2 * tol + 2.0 ** -4 * 1.001 * want.abs() + 2.0 ** -10 * top / 448 * 1.001).all()
    want, tol = paged_plain.attention(held, a.q.cpu(), range(T + 1), a.dim ** -0.5, window, sinks)
    got = layer.attn.cpu().double().view(T, a.Hq, a.dim)
    assert ((got - want).abs() <= tol).all()


def test_the_step_as_a_graph(example):
    T, D = 4, 256
    layers = [example.MixedLayer(T, D, 128, 8, 2, 256, attention=example.Attention(T, D, 100)) for _ in range(2)]
    for layer in layers:
        for p in (*layer.attention.pages, *layer.attention.scales.values()):
            p.view(torch.uint8).zero_()
        layer.attention.prompt(torch.ones(T, 9, D, device="cuda").bfloat16())
    eager, graphed = layers
    graph = graphed.capture()  # one eager step before it
    eager.step()
    for rep in range(5):
        for layer in layers:
            layer.attention.x.mul_(-1.5)
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert graphed.attention.lengths.tolist() == eager.attention.lengths.tolist() == [11 + rep] * T
        assert torch.equal(eager.attn, graphed.attn) and torch.equal(eager.y, graphed.y), rep
