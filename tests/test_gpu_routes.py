"""The calls of tests/operator_routes.py, each of which reaches a certain kernel, against float64; what must not leave its row or Y,
for every shape of the 8-bit product; the router for many tokens.

Bounds as in test_gpu_fp8.py and test_gpu_moe.py, where they are derived. The router's are those of test_gpu_moe.py with the
float64 logits computed on the GPU.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import microscaling_fp4_quantized_amd as F
import moe_plain as P
import operator_routes as R
from parity import say
from test_gpu_fp8 import check_linear, random_operands
from test_gpu_moe import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("M,N,K", [c for cases in R.LINEAR.values() for c in cases])
def test_linear(M, N, K):
    check_linear(M, N, K)


@pytest.mark.parametrize("shape", sorted(R.EDGES))
def test_linear_writes_its_rows_and_nothing_past_them(shape):
    M, N, K = R.EDGES[shape]
    (xq, xs, wq, ws), y = check_linear(M, N, K)
    guard = torch.full((M * N + 40000,), 7.0, dtype=torch.bfloat16, device=DEV)
    guard[:M * N] = float("nan")
    F.fp8_linear(xq, xs, wq, ws, out=guard[:M * N].view(M, N))
    assert torch.equal(guard[:M * N].view(M, N), y) and bool((guard[M * N:] == 7.0).all())


@pytest.mark.parametrize("shape", sorted(R.EDGES))
def test_linear_non_finite_stay_in_their_rows(shape):
    M, N, K = R.EDGES[shape]
    say(f"fp8_linear with NaN, M {M} N {N} K {K}")
    xq, xs, wq, ws = random_operands(np.random.default_rng(shape), M, N, K)
    clean = F.fp8_linear(xq, xs, wq, ws)
    rows, cols, band = [M // 2, M - 1], [5, N - 1], N // 128 // 2
    xs[rows[0], 1] = float("nan")
    xq.view(torch.uint8)[rows[1], K - 1] = 0x7F  # the NaN code
    wq.view(torch.uint8)[cols[0], 100] = 0x7F
    wq.view(torch.uint8)[cols[1], K - 3] = 0xFF
    ws[band, 2] = float("inf")  # of 128 features: infinite or, where a block's sum is 0, NaN
    y = F.fp8_linear(xq, xs, wq, ws)
    bad = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    bad[rows], bad[:, cols] = True, True
    assert bool(torch.isnan(y[bad]).all())
    bad[:, band * 128:band * 128 + 128] = True
    assert not bool(torch.isfinite(y[bad]).any())
    assert torch.equal(y[~bad], clean[~bad])


def ids_of(rng, T, k, E, loads):
    """[T, k] ids in which len(loads) of the E experts stand loads[i] times each, the other slots unused."""
    ids = np.full(T * k, -1)
    used = np.sort(rng.permutation(E)[:len(loads)])
    ids[rng.permutation(T * k)[:sum(loads)]] = np.repeat(used, loads)
    return ids.reshape(T, k), used


@pytest.mark.parametrize("T,k,E,D,I,block,up,down,loads", R.EXPERTS)
def test_experts(T, k, E, D, I, block, up, down, loads):
    say(f"experts T {T} E {E} D {D} I {I} k {k} block {block}: {up} and {down} waves")
    rng = np.random.default_rng(D + I + T)
    gen = torch.Generator(DEV).manual_seed(D + I + T)

    def codes(*shape):
        return torch.randint(0, 256, shape, dtype=torch.uint8, device=DEV, generator=gen)

    def scales(*shape):
        return torch.randint(118, 126, shape, dtype=torch.uint8, device=DEV, generator=gen)

    w13, w2 = (codes(E, 2 * I, D // 2), scales(E, 2 * I, D // 32)), (codes(E, D, I // 2), scales(E, D, I // 32))
    x = torch.randn(T, D, device=DEV, generator=gen).bfloat16()
    ids, used = ids_of(rng, T, k, E, loads)
    weights = rng.random((T, k)).astype(np.float32)
    y = F.fp4_moe_experts(x, torch.from_numpy(ids.astype(np.int32)).to(DEV), torch.from_numpy(weights).to(DEV), *w13, *w2, block)
    # the used experts alone, renumbered
    plain = [P.matrix(q[used].cpu().numpy(), s[used].cpu().numpy()) for q, s in (w13, w2)]
    ref, size = P.experts(f64(x), np.where(ids < 0, -1, np.searchsorted(used, ids)), weights, *plain, block)
    tol = 2.0 ** -8.8 * size
    tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.all(np.abs(f64(y) - ref) <= tol)
    over = (np.linalg.norm(f64(y) - ref) - np.linalg.norm(f64(torch.from_numpy(ref).bfloat16()) - ref)) / np.linalg.norm(ref)
    say(f"  norm error over the rounding's {over:.2e}")
    assert over <= 4.6e-4
    assert (f64(y)[(ids < 0).all(1)] == 0).all()


@pytest.mark.parametrize("T,E,D,k", [(399, 256, 3200, 8), (4099, 100, 1152, 6), (65537, 16, 256, 4), (1048560, 3, 128, 2)])
def test_route_of_many_tokens(T, E, D, k):
    say(f"route T {T} E {E} D {D} k {k}")
    gen = torch.Generator(DEV).manual_seed(T)
    x = torch.randn(T, D, device=DEV, generator=gen).bfloat16()
    w = (torch.randn(E, D, device=DEV, generator=gen) / D ** 0.5).bfloat16()
    ids, p = F.fp4_moe_route(x, w, k, renormalize=False)
    z = x.double() @ w.double().t()
    d = (np.log2(D) + 8) * 2.0 ** -24 * (x.double().abs() @ w.double().abs().t()).amax(1)
    at = ids.long()
    assert bool(((at >= 0) & (at < E)).all()) and bool((at.sort(1)[0].diff(dim=1) > 0).all())
    chosen = z.gather(1, at)
    assert bool((chosen >= z.topk(k, dim=1)[0] - 2 * d[:, None]).all())
    want = torch.softmax(z, 1).gather(1, at)
    assert bool(((p.double() - want).abs() <= (2 * d[:, None] + 1e-6) * want).all())


@pytest.mark.parametrize("T,E,k", [(3, 8, 2), (96, 8, 6)])
def test_experts_token_without_a_used_slot_gets_zeros_whatever_it_holds(T, E, k):
    """In two launches and in five."""
    D, I = 1024, 256
    say(f"experts T {T}: no slot of a NaN token used")
    gen = torch.Generator(DEV).manual_seed(T)
    w = [torch.randint(0, 256, (E, 2 * I, D // 2), dtype=torch.uint8, device=DEV, generator=gen),
         torch.randint(118, 126, (E, 2 * I, D // 32), dtype=torch.uint8, device=DEV, generator=gen),
         torch.randint(0, 256, (E, D, I // 2), dtype=torch.uint8, device=DEV, generator=gen),
         torch.randint(118, 126, (E, D, I // 32), dtype=torch.uint8, device=DEV, generator=gen)]
    x, p = torch.randn(T, D, device=DEV, generator=gen).bfloat16(), torch.rand(T, k, device=DEV, generator=gen)
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device=DEV, generator=gen)
    ids[1] = -1
    want = F.fp4_moe_experts(x, ids, p, *w, 32)
    x[1] = float("nan")
    y = F.fp4_moe_experts(x, ids, p, *w, 32)
    assert bool((y[1] == 0).all()) and torch.equal(y.view(torch.int16), want.view(torch.int16))
