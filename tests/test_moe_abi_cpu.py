"""Argument validation of the mixture-of-experts operators, in the library and in the Python calls: bad calls are
refused before anything touches a GPU."""
import os

import pytest
import torch

import microscaling_fp4_quantized_amd as F
from microscaling_fp4_quantized_amd import binding

A16 = 0x10000  # a 16-byte aligned fake address: never dereferenced, validation fails first
NULLPTR, SHAPE, BLOCK, ALIGN = -1, -2, -3, -5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        pytest.skip("libfp4.so not built")
    return binding.load_library()


def test_route_validation(lib):
    def r(X=A16, T=4, D=256, ld=256, W=A16, E=16, k=2, ids=A16, weights=A16, ws=A16, n=4 * 4 * 16 * 4):
        return lib.fp4_moe_route(X, T, D, ld, W, E, k, 1, ids, weights, ws, n, None)

    assert r(X=None) == r(W=None) == r(ids=None) == r(weights=None) == r(ws=None) == NULLPTR
    assert r(T=0) == r(T=-1) == r(D=0, ld=0) == r(D=64) == r(D=192) == r(D=(1 << 24) + 128, ld=1 << 25) == SHAPE
    assert r(E=0) == r(E=1025, n=1 << 20) == r(T=1 << 31, n=1 << 40) == r(T=16 * 65535 + 1, n=1 << 40) == SHAPE
    assert r(k=0) == r(k=-1) == r(k=17, E=32, n=1 << 20) == r(k=17) == r(k=3, E=2) == SHAPE
    assert r(ld=128) == r(ld=(1 << 40) + 8) == r(n=4 * 4 * 16 * 4 - 1) == SHAPE
    assert r(X=A16 + 2) == r(ld=260) == r(W=A16 + 8) == r(ws=A16 + 4) == r(ids=A16 + 2) == r(weights=A16 + 1) == ALIGN
    assert b"fp4_moe_route" in lib.fp4_last_error()


def test_experts_validation(lib):
    need = binding.moe_workspace_bytes(4, 2, 256, 128)

    def e(X=A16, T=4, D=256, ld=256, ids=A16, weights=A16, k=2, E=8, I=128, block=32, w13q=A16, w13s=A16, w2q=A16,
          w2s=A16, Y=A16, ws=A16, n=need):
        return lib.fp4_moe_experts(X, T, D, ld, ids, weights, k, E, I, block, w13q, w13s, w2q, w2s, Y, ws, n, None)

    assert e(block=0) == e(block=8) == e(block=48) == e(block=256) == e(block=-32) == BLOCK
    assert e(X=None) == e(ids=None) == e(weights=None) == e(w13q=None) == e(w13s=None) == NULLPTR
    assert e(w2q=None) == e(w2s=None) == e(Y=None) == e(ws=None) == NULLPTR
    assert e(T=0) == e(T=129, n=1 << 40) == e(k=0) == e(k=17, n=1 << 40) == SHAPE
    assert e(E=0) == e(E=1025) == e(D=64, ld=64) == e(D=320, ld=320, n=1 << 30) == e(I=0) == e(I=64) == SHAPE
    assert e(D=65536 + 128, ld=1 << 17, n=1 << 40) == e(I=65536 + 128, n=1 << 40) == SHAPE
    assert e(ld=128) == e(ld=(1 << 40) + 8) == e(n=need - 1) == SHAPE
    assert e(X=A16 + 2) == e(ld=260) == e(w13q=A16 + 8) == e(w13s=A16 + 4) == e(w2q=A16 + 1) == e(w2s=A16 + 8) == ALIGN
    assert e(Y=A16 + 8) == e(ws=A16 + 8) == e(ids=A16 + 2) == e(weights=A16 + 2) == ALIGN
    assert b"fp4_moe_experts" in lib.fp4_last_error()


def test_python_calls_refuse_what_the_kernels_cannot_take():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.zeros(8, 256, dtype=torch.bfloat16)
    ids, p = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    w13q, w13s = torch.zeros(8, 256, 128, dtype=torch.uint8), torch.zeros(8, 256, 8, dtype=torch.uint8)
    w2q, w2s = torch.zeros(8, 256, 64, dtype=torch.uint8), torch.zeros(8, 256, 4, dtype=torch.uint8)
    for call in (lambda: F.fp4_moe_route(x, w, 2), lambda: F.fp4_moe_route(x, w[0], 2),
                 lambda: F.fp4_moe_route(x, None, 2), lambda: F.fp4_moe_route(x.float(), w, 2),
                 lambda: F.fp4_moe_experts(x, ids, p, w13q, w13s, w2q, w2s, 32),
                 lambda: F.fp4_moe_experts(None, ids, p, w13q, w13s, w2q, w2s, 32),
                 lambda: F.fp4_moe_experts(x, ids, p, w13q[0], w13s, w2q, w2s, 32)):
        with pytest.raises(ValueError):
            call()


def test_workspace_bytes_of_both_sides_agree(lib):
    """The library refuses one byte less than moe_workspace_bytes says and does not refuse that much for its size."""
    for T, k, D, I in ((1, 1, 128, 128), (3, 5, 384, 640), (128, 16, 65536, 65536), (64, 6, 4096, 1408)):
        n = binding.moe_workspace_bytes(T, k, D, I)

        def call(size, y):
            return lib.fp4_moe_experts(A16, T, D, D, A16, A16, k, 8, I, 32, A16, A16, A16, A16, y, A16, size, None)
        assert call(n - 1, A16) == SHAPE and call(n, A16 + 8) == ALIGN  # sizes are checked before alignment
