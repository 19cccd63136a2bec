"""Mixture-of-experts operators on the GPU against float64.

Router: products of bf16 are exact in float32 and a logit is a sum of D of them in float32 in some order, so it is
off by at most (log2(D) + 8) * 2^-24 * sum |x w| for sums in blocks of up to 256; call that d (the largest of a token).
A chosen expert's float64 logit is at least the k-th largest minus 2 d, a weight is within 2 d + 1e-6 (exp, sum and
division in float32) relative of the float64 softmax.

Experts: activations enter with a relative error of 2^-12 of themselves or 2^-18 of their group's largest, the
matrix cores cut products 13 bits below the largest of their eight: 2^-12 + 7 * 2^-13 < 2^-9.8 of the sum of
magnitudes behind every value in the worst case, twice (x and h). size below carries those magnitudes through both
products (a bound; the errors are random, so most are far below): |error| <= 2^-8.8 * size + half a bf16 step.
In norm the errors are random: the terms leave at most 2^-12 / sqrt(3) of x and of h, the cut products 1.4e-5 of each
product's result, together e = 2.3e-4 of y before its rounding, and rounding y + e instead of y takes it at most 2 e further
from y than y's own rounding does: ||out - y|| <= ||bf16(y) - y|| + 4.6e-4 ||y||.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import microscaling_fp4_quantized_amd as F
import moe_plain as P
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda"


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16().to(DEV)


def f64(t):
    return t.detach().cpu().double().numpy()


ROUTE = [(1, 8, 128, 1), (1, 128, 2048, 8), (3, 1, 256, 1), (5, 60, 512, 6), (16, 64, 1024, 16), (17, 100, 4096, 8),
         (61, 256, 4096, 6), (130, 1024, 256, 16), (500, 17, 7168, 3)]


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,D,k", ROUTE)
def test_route(T, E, D, k, renormalize):
    say(f"route T {T} E {E} D {D} k {k}")
    rng = np.random.default_rng(T + E + D)
    big = bf16(rng.standard_normal((T, D + 8)))
    x, w = big[:, :D], bf16(rng.standard_normal((E, D)) / np.sqrt(D))
    ids, p = F.fp4_moe_route(x, w, k, renormalize=renormalize)
    assert ids.dtype == torch.int32 and p.dtype == torch.float32 and ids.shape == p.shape == (T, k)
    ids, p = ids.cpu().numpy(), f64(p)
    z, soft = P.route(f64(x), f64(w))
    d = (np.log2(D) + 8) * 2.0 ** -24 * (np.abs(f64(x)) @ np.abs(f64(w)).T).max(1)
    assert ids.min() >= 0 and ids.max() < E
    assert all(len(set(row)) == k for row in ids)
    zc = np.take_along_axis(z, ids, 1)
    assert np.all(zc >= np.sort(z, 1)[:, ::-1][:, :k] - 2 * d[:, None])
    want = np.take_along_axis(soft, ids, 1)
    if renormalize:
        want = want / want.sum(1, keepdims=True)
    err = np.abs(p - want) / want
    say(f"  worst {np.max(err / (2 * d[:, None] + 1e-6)):.3f} of the bound")
    assert np.all(err <= 2 * d[:, None] + 1e-6)


def test_route_ties_zeros_and_nan():
    T, E, D = 6, 70, 256
    x = torch.zeros(T, D, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(E, D, dtype=torch.bfloat16, device=DEV)
    x[1:, 0] = 1
    w[:, 0] = 0.5
    w[[65, 3, 40], 0] = 2.0
    x[3, 0] = -1.0
    x[4, 5] = float("nan")
    ids, p = F.fp4_moe_route(x, w, 5)
    ids = ids.cpu().numpy()
    assert ids[0].tolist() == [0, 1, 2, 3, 4]           # all equal
    assert ids[1].tolist() == [3, 40, 65, 0, 1]         # three equal, then the rest in order
    assert ids[3].tolist() == [0, 1, 2, 4, 5]           # the three are now the smallest
    assert len(set(ids[4])) == 5 and torch.isnan(p[4]).all()
    assert torch.isfinite(p[[0, 1, 2, 3, 5]]).all()
    assert torch.allclose(p[0], torch.full((5,), 0.2, device=DEV))


def mxfp4(rng, *shape, std=0.05):
    """MXFP4 matrices from bf16 weights through the framework's quantizer is another test; here random codes."""
    codes = rng.integers(0, 256, (*shape[:-1], shape[-1] // 2), dtype=np.uint8)
    scales = rng.integers(118, 126, (*shape[:-1], shape[-1] // 32), dtype=np.uint8)
    return codes, scales


def run_experts(T, E, D, I, k, block, ids=None, x=None, seed=0, more=0):
    say(f"experts T {T} E {E} D {D} I {I} k {k} block {block}")
    rng = np.random.default_rng(seed + T + E + D + I)
    w13, w2 = mxfp4(rng, E, 2 * I, D), mxfp4(rng, E, D, I)
    if x is None:
        x = bf16(rng.standard_normal((T, D + more)))[:, :D]
    if ids is None:
        ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    weights = rng.random(ids.shape).astype(np.float32)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    args = (x, t(ids.astype(np.int32)), t(weights), t(w13[0]), t(w13[1]), t(w2[0]), t(w2[1]), block)
    y = F.fp4_moe_experts(*args)
    assert y.shape == (T, D) and y.dtype == torch.bfloat16
    return args, y, (f64(x), ids, weights, P.matrix(*w13), P.matrix(*w2), block)


def check_experts(*a, **kw):
    args, y, plain = run_experts(*a, **kw)
    ref, size = P.experts(*plain)
    tol = 2.0 ** -8.8 * size
    tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(f64(y) - ref)
    assert np.all(err <= tol)
    norm = max(np.linalg.norm(ref), 1e-300)
    over = (np.linalg.norm(f64(y) - ref) - np.linalg.norm(f64(torch.from_numpy(ref).bfloat16()) - ref)) / norm
    say(f"  norm error over the rounding's {over:.2e}")
    assert over <= 4.6e-4
    return args, y


EXPERTS = [(1, 1, 128, 128, 1, 32), (1, 8, 256, 128, 2, 16), (1, 16, 2048, 768, 8, 32), (2, 4, 128, 384, 4, 128),
           (3, 6, 640, 256, 3, 64), (4, 4, 1152, 128, 2, 32), (7, 3, 512, 640, 3, 128), (16, 8, 384, 256, 2, 16),
           (33, 4, 256, 128, 2, 32), (64, 16, 256, 256, 4, 64), (128, 2, 128, 128, 1, 32), (128, 3, 256, 128, 2, 128),
           (5, 40, 4096, 128, 2, 32), (2, 3, 128, 2048, 2, 64), (3, 2, 4224, 128, 1, 32), (2, 3, 7168, 256, 2, 128),
          (2, 2, 128, 4352, 1, 64), (6, 3, 8320, 128, 2, 16), (12, 2, 1408, 1408, 1, 128)]


@pytest.mark.parametrize("T,E,D,I,k,block", EXPERTS)
def test_experts(T, E, D, I, k, block):
    check_experts(T, E, D, I, k, block, more=8 * (T % 3))


# Work enough that pairs are sorted by expert and an expert's matrices are read once for all of its tokens (at least 75 MB
# if every pair read its own): one token an expert to all of them on one; rows of scales longer than LDS holds at
# once; K of whole and of half slices; enough tiles for small workgroups in one product, the other and neither
SORTED = [(128, 16, 256, 128, 16, 32), (128, 16, 128, 256, 16, 16), (100, 20, 384, 640, 8, 64),
          (64, 16, 1152, 128, 8, 128), (37, 9, 4224, 128, 7, 32), (19, 5, 128, 4352, 5, 64), (50, 12, 7168, 256, 3, 128),
          (24, 3, 8320, 128, 3, 16), (12, 4, 1408, 1408, 2, 128), (128, 60, 640, 256, 3, 64), (90, 32, 256, 1024, 5, 32),
          (128, 64, 1024, 128, 4, 64), (20, 32, 2048, 1664, 2, 32), (60, 64, 512, 1152, 3, 16)]


@pytest.mark.parametrize("T,E,D,I,k,block", SORTED)
def test_experts_sorted(T, E, D, I, k, block):
    check_experts(T, E, D, I, k, block, more=8 * (T % 3))


def test_experts_sorted_all_tokens_on_one_expert_of_many():
    check_experts(128, 120, 2048, 128, 2, 32, ids=np.full((128, 2), 119))


def test_experts_sorted_unused_slots_and_non_finite_tokens():
    T, E, D, k = 96, 8, 1024, 6
    rng = np.random.default_rng(12)
    ids = rng.integers(-3, E + 2, (T, k))
    ids[5] = -1
    x = bf16(rng.standard_normal((T, D)))
    args, y = check_experts(T, E, D, 256, k, 32, ids=ids, x=x)
    assert (y[5] == 0).all()
    sick = x.clone()
    ids[[7, 40], 0] = 0
    sick[7, 100] = float("nan")
    sick[40, 900] = -float("inf")
    _, y, _ = run_experts(T, E, D, 256, k, 32, ids=ids, x=x)
    _, z, _ = run_experts(T, E, D, 256, k, 32, ids=ids, x=sick)
    assert torch.isnan(z[[7, 40]]).all()
    rest = [t for t in range(T) if t not in (7, 40)]
    assert torch.equal(z[rest].view(torch.int16), y[rest].view(torch.int16))


def test_experts_unused_slots_and_repeated_experts():
    ids = np.array([[-1, -1, -1], [2, 2, 2], [0, -1, 0], [5, 7, 1 << 30], [-5, 3, 4], [1, 0, 1]])
    args, y = check_experts(6, 5, 256, 128, 3, 32, ids=ids)
    assert (y[0] == 0).all()
    # the weight of an unused slot may be anything
    w = args[2].clone()
    w[0, 1] = float("nan")
    w[3, 2] = float("inf")
    again = F.fp4_moe_experts(args[0], args[1], w, *args[3:])
    assert torch.equal(again.view(torch.int16), y.view(torch.int16))


def test_experts_all_tokens_on_one_expert_of_many():
    ids = np.full((128, 1), 999)
    check_experts(128, 1000, 128, 128, 1, 32, ids=ids)


@pytest.mark.parametrize("scale", [0.0, 1e-38, 1e-20, 1e12])
def test_experts_ranges(scale):
    """Inputs far from 1 keep the relative accuracy; zeros give zeros."""
    rng = np.random.default_rng(9)
    x = bf16(rng.standard_normal((3, 256)) * scale)
    if scale in (0.0, 1e-38):  # below the code's floor the terms vanish gradually; y is 0 in bf16 either way
        _, y, _ = run_experts(3, 4, 256, 128, 2, 32, x=x)
        assert (y == 0).all()
    elif scale < 1:            # h is quadratic in x: y is far below bf16's smallest number of note, but finite
        _, y, _ = run_experts(3, 4, 256, 128, 2, 32, x=x)
        assert torch.isfinite(y).all()
    else:
        check_experts(3, 4, 256, 128, 2, 32, x=x)


def test_experts_non_finite_tokens_stay_alone():
    rng = np.random.default_rng(10)
    x = bf16(rng.standard_normal((8, 256)))
    clean = x.clone()
    x[2, 7] = float("nan")
    x[5, 200] = float("inf")
    ids = np.tile(np.array([[0, 1]]), (8, 1))
    args, y, _ = run_experts(8, 2, 256, 128, 2, 32, ids=ids, x=x)
    _, y0, _ = run_experts(8, 2, 256, 128, 2, 32, ids=ids, x=clean)
    assert torch.isnan(y[2]).all() and torch.isnan(y[5]).all()
    rest = [0, 1, 3, 4, 6, 7]
    assert torch.equal(y[rest].view(torch.int16), y0[rest].view(torch.int16))


def test_experts_with_quantized_weights_follow_the_dense_layer():
    """Weights through fp4_quantize_weights: against the dense layer on the unrotated bf16 weights, the result is off by
    the MXFP4 rounding of three matrices, about 2^-3.5 each in norm, so well within 0.5."""
    rng = np.random.default_rng(11)
    T, E, D, I, k, block = 9, 4, 512, 256, 2, 32
    W13, W2 = bf16(rng.standard_normal((E * 2 * I, D)) * 0.05), bf16(rng.standard_normal((E * D, I)) * 0.05)
    q13, q2 = F.fp4_quantize_weights(W13, block), F.fp4_quantize_weights(W2, block)
    x, wr = bf16(rng.standard_normal((T, D))), bf16(rng.standard_normal((E, D)) / 20)
    ids, p = F.fp4_moe_route(x, wr, k)
    y = F.fp4_moe_experts(x, ids, p, q13[0].view(E, 2 * I, D // 2), q13[1].view(E, 2 * I, D // 32),
                          q2[0].view(E, D, I // 2), q2[1].view(E, D, I // 32), block)
    w13, w2 = f64(W13).reshape(E, 2 * I, D), f64(W2).reshape(E, D, I)
    ref = np.zeros((T, D))
    for t in range(T):
        for e, w in zip(ids.cpu().numpy()[t], f64(p)[t]):
            u = w13[e] @ f64(x)[t]
            ref[t] += w * (w2[e] @ (u[:I] / (1 + np.exp(-u[:I])) * u[I:]))
    rel = np.linalg.norm(f64(y) - ref) / np.linalg.norm(ref)
    say(f"  against the dense layer {rel:.3f}")
    assert rel < 0.5


def test_experts_same_bits_again_and_in_given_buffers():
    args, y, _ = run_experts(20, 6, 384, 256, 3, 64)
    ws = torch.full((F.moe_workspace_bytes(20, 3, 384, 256) + 1,), 255, dtype=torch.uint8, device=DEV)
    guard = torch.full((20 * 384 + 512,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = F.fp4_moe_experts(*args, out=guard[:20 * 384].view(20, 384), workspace=ws)
    assert torch.equal(out.view(torch.int16), y.view(torch.int16))
    assert (guard[20 * 384:] == 7.0).all() and ws[-1] == 255
