"""The mixed-precision layer of examples/: each of its stages against float64 on that stage's own inputs, and its graph
against the eager step.

Bounds: a bf16 result is half a step off, 2^-9 in norm at most; 8-bit products add 1.4e-5, experts 4.6e-4 over that; a norm's
float32 sums and its codes' inputs add less than 2^-16. So 2^-8 of the result in norm holds for every stage.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import fp8_plain
import moe_plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixed_layer.py")
    spec = importlib.util.spec_from_file_location("mixed_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def f64(t):
    return t.detach().cpu().double().numpy()


def near(got, want):
    assert np.linalg.norm(f64(got) - want) <= 2.0 ** -8 * np.linalg.norm(want)


@pytest.mark.parametrize("T,D,I,E,k,N", [(1, 256, 128, 8, 2, 640), (21, 384, 256, 5, 3, 130)])
def test_layer(example, T, D, I, E, k, N):
    layer = example.MixedLayer(T, D, I, E, k, N)
    y = layer.step()
    torch.cuda.synchronize()
    proj, head = (fp8_plain.values(*w, 128) for w in (layer.proj, layer.head))
    near(layer.o, fp8_plain.values(*layer.attn8, 1) @ proj.T)
    h, n = fp8_plain.rmsnorm(f64(layer.o), f64(layer.hidden), f64(layer.norm1), 1e-6)
    near(layer.n1[2], h)
    near(layer.n1[3], n)
    w13, w2 = (moe_plain.matrix(q.cpu().numpy(), s.cpu().numpy()) for q, s in (layer.experts[:2], layer.experts[2:]))
    ids, p = layer.routed
    moe, _ = moe_plain.experts(f64(layer.n1[3]), ids.cpu().numpy(), f64(p), w13, w2, layer.block)
    near(layer.moe, moe)
    h2, _ = fp8_plain.rmsnorm(f64(layer.moe), f64(layer.n1[2]), f64(layer.norm2), 1e-6)
    near(layer.n2[2], h2)
    near(y, fp8_plain.values(*layer.n2[:2], 1) @ head.T)

    want = y.clone()
    graph = layer.capture()
    attn = layer.attn.clone()
    for rep in range(4):
        layer.attn.copy_(-attn.flip(0) * 2)  # another step, eagerly, on the same buffers
        layer.step()
        torch.cuda.synchronize()
        assert not torch.equal(layer.y, want)
        layer.attn.copy_(attn)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.y, want), rep
