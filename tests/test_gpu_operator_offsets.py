"""The 8-bit and mixture-of-experts operators where offsets pass 2^31 elements and 2^32 bytes: the far end of a large operand gives what
it gives as an operand of its own.

Rows and features are independent, so quantized rows are equal bit for bit, and so are products and experts up to the
order of float32 sums, which may go by the operand's size: both sides are then one rounding to bf16 (2^-9 at most) of nearly
equal sums, so they agree within 2^-8 in norm.
"""
import pytest
import torch

import microscaling_fp4_quantized_amd as F
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda"


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def near(a, b):
    a, b = a.double(), b.double()
    return bool((a - b).norm() <= 2.0 ** -8 * b.norm()) and bool(b.norm() > 0)


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def normal(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(shape[0]))


def test_rows_past_2_31_elements():
    M, K, end = (1 << 31) // 4096 + 133, 4096, 67
    say(f"quantize {M} x {K}")
    x = normal(M, K)
    c, s = F.fp8_quantize(x)
    tail = x[-end:].clone()
    ct, st = F.fp8_quantize(tail)
    assert same(c[-end:], ct) and same(s[-end:], st)
    del c, s
    g = normal(K)
    out = F.fp8_add_rmsnorm_quantize(x, g, residual=x, normed=True)
    for a, b in zip(out, F.fp8_add_rmsnorm_quantize(tail, g, residual=tail, normed=True)):
        assert same(a[-end:], b)
    del out
    c, s = F.fp8_quantize_weights(x)
    block = M // 128 * 128 - 128  # the last whole block of rows, and those after it
    ct, st = F.fp8_quantize_weights(x[block:].clone())
    assert same(c[block:], ct) and same(s[block // 128:], st)


@pytest.mark.parametrize("M", [1, 20, 300])
def test_linear_with_weights_past_2_32_bytes(M):
    N, K = 600 * 1024 + 36, 8192
    say(f"linear {M} x {N} x {K}")
    w = torch.randint(0, 0x70, (N, K), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)  # finite, positive
    ws = torch.rand((N + 127) // 128, K // 128, device=DEV)
    xq, xs = F.fp8_quantize(normal(M, K))
    y = F.fp8_linear(xq, xs, w, ws)
    cut = N // 128 * 128 - 256
    assert near(y[:, cut:], F.fp8_linear(xq, xs, w[cut:].clone(), ws[cut // 128:].clone()))
    assert near(y[:, :512], F.fp8_linear(xq, xs, w[:512].clone(), ws[:4].clone()))


def test_linear_with_rows_past_2_31_elements():
    M, N, K = (1 << 31) // 2048 + 70, 2056, 256
    say(f"linear {M} x {N} x {K}")
    xq, xs = F.fp8_quantize(normal(M, K))
    w, ws = F.fp8_quantize_weights(normal(N, K))
    y = F.fp8_linear(xq, xs, w, ws)
    assert y.numel() > 1 << 31
    assert near(y[-130:], F.fp8_linear(xq[-130:].clone(), xs[-130:].clone(), w, ws))


@pytest.mark.parametrize("T,k", [(1, 4), (64, 6)])
def test_experts_past_2_32_bytes(T, k):
    E, D, I, keep = 800, 4096, 1408, 8
    say(f"experts T {T} of {E} of {D} x {I}")
    parts = [torch.randint(0, 256, (E, 2 * I, D // 2), dtype=torch.uint8, device=DEV),
             torch.randint(118, 124, (E, 2 * I, D // 32), dtype=torch.uint8, device=DEV),
             torch.randint(0, 256, (E, D, I // 2), dtype=torch.uint8, device=DEV),
             torch.randint(118, 124, (E, D, I // 32), dtype=torch.uint8, device=DEV)]
    assert parts[0].numel() > 1 << 32
    x, p = normal(T, D), torch.rand(T, k, device=DEV)
    ids = torch.randint(0, keep, (T, k), dtype=torch.int32, device=DEV)
    y = F.fp4_moe_experts(x, ids + (E - keep), p, *parts, 32)
    assert near(y, F.fp4_moe_experts(x, ids, p, *[t[-keep:].clone() for t in parts], 32))


def test_strides_past_2_31():
    """A few rows of a very wide buffer."""
    K, ld = 512, (1 << 30) + 64
    big = torch.zeros(3 * ld, dtype=torch.bfloat16, device=DEV)
    x = big.as_strided((3, K), (ld, 1))
    x.copy_(normal(3, K))
    own = x.contiguous()
    assert all(same(a, b) for a, b in zip(F.fp8_quantize(x), F.fp8_quantize(own)))
    g, w = normal(K), normal(12, K)
    assert all(same(a, b) for a, b in zip(F.fp8_add_rmsnorm_quantize(x, g, residual=x)[:3],
                                          F.fp8_add_rmsnorm_quantize(own, g, residual=own)[:3]))
    assert all(same(a, b) for a, b in zip(F.fp4_moe_route(x, w, 2), F.fp4_moe_route(own, w, 2)))
