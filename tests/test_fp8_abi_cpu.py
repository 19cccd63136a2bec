"""Argument validation of the 8-bit operators, in the library and in the Python calls: bad calls are refused
before anything touches a GPU."""
import os

import pytest
import torch

import microscaling_fp4_quantized_amd as F
from microscaling_fp4_quantized_amd import binding

A16 = 0x10000  # a 16-byte aligned fake address: never dereferenced, validation fails first
NULLPTR, SHAPE, ALIGN = -1, -2, -5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        pytest.skip("libfp4.so not built")
    return binding.load_library()


@pytest.mark.parametrize("name", ["fp8_quantize", "fp8_quantize_weights"])
def test_quantize_validation(lib, name):
    def q(X=A16, M=4, K=256, ld=256, codes=A16, scales=A16):
        return getattr(lib, name)(X, M, K, ld, codes, scales, None)

    assert q(X=None) == q(codes=None) == q(scales=None) == NULLPTR
    assert name.encode() in lib.fp4_last_error()
    assert q(M=0) == q(M=-1) == q(K=0, ld=0) == q(K=64) == q(K=192) == SHAPE
    assert q(ld=128) == q(ld=1 << 41) == SHAPE
    assert q(M=(1 << 31) // 32, K=256) == q(M=1 << 62, K=1 << 20, ld=1 << 20) == SHAPE
    assert q(X=A16 + 2) == q(ld=260) == q(codes=A16 + 8) == q(scales=A16 + 2) == ALIGN


def test_norm_validation(lib):
    def n(X=A16, M=4, K=256, ldx=256, r=A16, ldr=256, w=A16, eps=1e-6, codes=A16, scales=A16, h=2 * A16, y=None):
        return lib.fp8_add_rmsnorm_quantize(X, M, K, ldx, r, ldr, w, eps, codes, scales, h, y, None)

    assert n(X=None) == n(w=None) == n(codes=None) == n(scales=None) == NULLPTR
    assert n(r=None) == n(h=None) == NULLPTR  # the residual and its sum go together
    assert n(M=0) == n(K=200, ldx=200) == n(ldx=128) == n(ldr=128) == n(ldr=1 << 41) == SHAPE
    assert n(K=65536 + 128, ldx=1 << 17, ldr=1 << 17) == SHAPE
    assert n(eps=-1.0) == n(eps=float("nan")) == n(eps=float("inf")) == SHAPE
    assert n(h=A16, ldr=512) == SHAPE  # in place only without a gap between the rows
    assert n(r=A16 + 4) == n(ldr=260) == n(h=A16 + 4) == n(w=A16 + 8) == n(y=A16 + 2) == ALIGN
    assert b"fp8_add_rmsnorm_quantize" in lib.fp4_last_error()


def test_linear_validation(lib):
    def f(Xq=A16, Xs=A16, Wq=A16, Ws=A16, M=4, N=4, K=128, Y=A16):
        return lib.fp8_linear(Xq, Xs, Wq, Ws, M, N, K, Y, None)

    assert f(Xq=None) == f(Xs=None) == f(Wq=None) == f(Ws=None) == f(Y=None) == NULLPTR
    assert f(M=0) == f(N=0) == f(K=0) == f(K=64) == f(K=320) == SHAPE
    assert f(M=1 << 31) == f(N=1 << 31) == f(K=(1 << 23) + 128) == f(M=1 << 30, K=1 << 14) == SHAPE
    assert f(M=(1 << 31) - 1, N=(1 << 31) - 1) == SHAPE  # more tiles than a grid holds
    assert f(Xq=A16 + 8) == f(Wq=A16 + 4) == f(Y=A16 + 8) == f(Xs=A16 + 2) == f(Ws=A16 + 1) == ALIGN
    assert b"fp8_linear" in lib.fp4_last_error()


def test_python_calls_refuse_what_the_kernels_cannot_take():
    cpu = torch.zeros(4, 256, dtype=torch.bfloat16)
    for call in (lambda: F.fp8_quantize(cpu), lambda: F.fp8_quantize_weights(cpu), lambda: F.fp8_quantize(cpu[0]),
                 lambda: F.fp8_quantize(cpu.float()), lambda: F.fp8_quantize(cpu.t()),
                 lambda: F.fp8_add_rmsnorm_quantize(cpu, cpu[0]), lambda: F.fp8_linear(cpu, cpu, cpu, cpu),
                 lambda: F.fp8_linear(None, cpu, cpu, cpu)):
        with pytest.raises(ValueError):
            call()
