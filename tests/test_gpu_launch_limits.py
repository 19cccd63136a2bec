"""Calls of more work-items than one grid dimension holds (2^32): rows of 128 through the norm, and 8-bit products of very many
features or rows. Every output is written, and those at the ends are what a call of their own gives.

Rows and features are independent, so the norm's are equal bit for bit; a product's float32 sums may go in another order in a
smaller call, so both are one bf16 rounding (2^-9 at most) of nearly equal sums: within 2^-8 in norm.
"""
import pytest
import torch

import microscaling_fp4_quantized_amd as F
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN8 = 0x7F  # the NaN code


@pytest.fixture(autouse=True)
def _free():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def near(a, b):
    a, b = a.double(), b.double()
    return bool((a - b).norm() <= 2.0 ** -8 * b.norm()) and bool(b.norm() > 0)


def repeated(base, rows):
    """`rows` rows: base over and over."""
    out = torch.empty(rows, base.shape[1], dtype=base.dtype, device=DEV)
    whole = rows // base.shape[0] * base.shape[0]
    out[:whole].view(-1, *base.shape).copy_(base)
    out[whole:].copy_(base[:rows - whole])
    return out


def test_norm_of_2_26_rows_of_128():
    M, K, n = (1 << 26) + 4099, 128, 5000
    say(f"norm {M} x {K}")
    base = torch.empty(9973, K, dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(1))
    x, g = repeated(base, M), torch.ones(K, dtype=torch.bfloat16, device=DEV)
    codes = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=DEV)
    codes.view(torch.uint8).fill_(NAN8)
    scales = torch.full((M, 1), float("nan"), device=DEV)
    F.fp8_add_rmsnorm_quantize(x, g, out=(codes, scales, None, None))
    assert not torch.isnan(scales).any() and not (codes.view(torch.uint8) == NAN8).any()
    for rows in (slice(0, n), slice(M // 2, M // 2 + n), slice(M - n, M)):
        c, s, _, _ = F.fp8_add_rmsnorm_quantize(x[rows].clone(), g)
        assert same(codes[rows], c) and same(scales[rows], s)


def test_linear_of_2_28_features():
    M, N, K, n = 1, (1 << 28) + 2057, 128, 4096
    say(f"linear {M} x {N} x {K}")
    base = torch.randint(0, 0x70, (7919, K), dtype=torch.uint8, device=DEV)  # finite, positive
    w = repeated(base, N).view(torch.float8_e4m3fn)
    ws = torch.rand((N + 127) // 128, 1, device=DEV) + 0.5
    xq, xs = F.fp8_quantize(torch.randn(M, K, device=DEV).bfloat16())
    y = F.fp8_linear(xq, xs, w, ws, out=torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV))
    assert not torch.isnan(y).any()
    for a in (0, N // 256 * 128, N // 128 * 128 - n):
        b = min(N, a + 2 * n)
        assert near(y[:, a:b], F.fp8_linear(xq, xs, w[a:b].clone(), ws[a // 128:(b + 127) // 128].clone()))


def test_linear_of_2_28_rows():
    M, N, K, n = (1 << 28) + 1033, 3, 128, 4096
    say(f"linear {M} x {N} x {K}")
    base = torch.randint(0, 0x70, (7919, K), dtype=torch.uint8, device=DEV)
    xq, xs = repeated(base, M).view(torch.float8_e4m3fn), torch.rand(M, 1, device=DEV) + 0.5
    w, ws = F.fp8_quantize_weights(torch.randn(N, K, device=DEV).bfloat16())
    y = F.fp8_linear(xq, xs, w, ws, out=torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV))
    assert not torch.isnan(y).any()
    for a in (0, M // 2, M - n):
        assert near(y[a:a + n], F.fp8_linear(xq[a:a + n].clone(), xs[a:a + n].clone(), w, ws))
