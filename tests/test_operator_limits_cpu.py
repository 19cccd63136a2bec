"""The sizes that the library refuses are those that include/fp4.h names, and the message says which."""
import os
import re

import pytest

from microscaling_fp4_quantized_amd import binding

A16 = 0x10000  # a 16-byte aligned fake address: never dereferenced, validation fails first
SHAPE, ALIGN = -2, -5
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fp4.h")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        pytest.skip("libfp4.so not built")
    return binding.load_library()


def test_the_routers_tokens(lib):
    """Sizes are checked before alignment: a misaligned operand shows which sizes pass, without a launch."""
    with open(HEADER) as f:
        most = int(re.search(r"#define FP4_MOE_ROUTE_MAX_TOKENS (\d+)", f.read()).group(1))

    def r(T, E, ids=A16 + 2):
        return lib.fp4_moe_route(A16, T, 256, 256, A16, E, 1, 1, ids, A16, A16, 1 << 60, None)

    for E in (1, 16, 1024):
        assert r(most, E) == ALIGN
        assert r(most + 1, E) == SHAPE
        assert str(most).encode() in lib.fp4_last_error()


def test_any_finite_eps(lib):
    def n(eps, h=A16 + 4):  # the misaligned output is found after eps
        return lib.fp8_add_rmsnorm_quantize(A16, 4, 256, 256, A16, 256, A16, eps, A16, A16, h, None, None)

    assert n(0.0) == n(3.4028234e38) == ALIGN
    assert n(float("inf")) == n(float("nan")) == n(-1e-30) == SHAPE


def test_the_products_tiles(lib):
    def f(M, N, K=128, ws=A16 + 1):
        return lib.fp8_linear(A16, A16, A16, ws, M, N, K, A16, None)

    assert f((1 << 31) - 1, 128) == f(128, (1 << 31) - 1) == f(1, (1 << 31) - 1) == ALIGN
    assert f((1 << 31) - 1, 8192) == SHAPE  # 2^24 x 2^7 tiles of 128 x 64
