"""Argument validation of the paged cache's calls, in the library and in the Python calls: bad calls are refused before anything
touches a GPU."""
import ctypes
import os

import pytest
import torch

import microscaling_fp4_quantized_amd as F
from microscaling_fp4_quantized_amd import binding

A16 = 0x10000  # a 16-byte aligned fake address: never dereferenced, validation fails first
NULLPTR, SHAPE, FORMAT, ALIGN = -1, -2, -4, -5
FAR = (1 << 40) + 16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        pytest.skip("libfp4.so not built")
    return binding.load_library()


def cache(**other):
    c = dict(k=A16, v=A16, k_scales=None, v_scales=None, pages=9, page_stride=4 * 16 * 128, head_stride=16 * 128, token_stride=128,
             scale_page_stride=0, scale_head_stride=0, scale_token_stride=0, table=A16, table_stride=5, cols=5, lengths=A16, batch=3,
             dtype=0, heads=4, dim=128, page_size=16)
    if other.get("dtype") == 1:
        c.update(k_scales=A16, v_scales=A16, scale_page_stride=64, scale_head_stride=16, scale_token_stride=1)
    c.update(other)
    return ctypes.byref(binding._KvCache(**c))


def append(lib, c=None, starts=A16, T=7, K=A16, kr=512, kh=128, V=A16, vr=512, vh=128, Q=A16, qr=2048, qh=128, Hq=16, O=2 * A16,
           our=2048, oh=128, freqs=A16, rotated=128, pos=None, axes=None, n=0, **other):
    return lib.fp4_kv_append(cache(**other) if c is None else c, starts, T, K, kr, kh, V, vr, vh, Q, qr, qh, Hq, O, our, oh, freqs,
                             rotated, 0, pos, axes, n, None)


def decode(lib, c=None, Q=A16, qr=2048, qh=128, Hq=16, scale=0.1, window=0, sinks=0, O=A16, ws=A16, n=1 << 40, **other):
    return lib.fp4_attention_decode(cache(**other) if c is None else c, Q, qr, qh, Hq, scale, window, sinks, O, ws, n, None)


def prompt(lib, c=None, starts=A16, T=7, Q=A16, qr=2048, qh=128, Hq=16, scale=0.1, window=0, sinks=0, O=A16, ws=A16, n=1 << 40,
           **other):
    return lib.fp4_attention_prompt(cache(**other) if c is None else c, starts, T, Q, qr, qh, Hq, scale, window, sinks, O, ws, n, None)


@pytest.mark.parametrize("call,late", [(append, dict(V=A16 + 2)), (decode, dict(O=A16 + 4)), (prompt, dict(O=A16 + 4))])
def test_the_caches_validation(lib, call, late):
    """`late` is refused last: with it a cache that passes shows as ALIGN."""
    def c(**other):
        return call(lib, **late, **other)

    assert call(lib, c=ctypes.POINTER(binding._KvCache)()) == NULLPTR
    assert c(k=None) == c(v=None) == c(table=None) == c(lengths=None) == NULLPTR
    assert c(k_scales=A16) == c(v_scales=A16) == c(dtype=1, k_scales=None) == c(dtype=1, v_scales=None) == NULLPTR
    assert c(dtype=2) == c(dtype=-1) == FORMAT
    assert c(heads=0) == c(heads=-4) == c(heads=1025) == c(dim=0) == c(dim=96) == c(dim=512) == SHAPE
    assert c(page_size=8) == c(page_size=0) == c(page_size=48) == c(page_size=2048) == SHAPE
    assert c(pages=0) == c(pages=1 << 31) == c(page_stride=64) == c(head_stride=0) == c(token_stride=FAR) == SHAPE
    assert c(token_stride=(1 << 25) + 16) == c(head_stride=FAR) == SHAPE and c(token_stride=1 << 25) == ALIGN
    assert c(dtype=1, scale_page_stride=0) == c(dtype=1, scale_token_stride=-1) == c(dtype=1, scale_head_stride=FAR) == SHAPE
    assert c(cols=0) == c(cols=6) == c(cols=(1 << 26) + 1, table_stride=1 << 27) == c(table_stride=FAR) == SHAPE
    assert c(batch=0) == c(batch=65536) == c(batch=33, cols=1 << 26, table_stride=1 << 26) == SHAPE
    assert c(k=A16 + 8) == c(v=A16 + 4) == c(page_stride=4 * 16 * 128 + 4) == c(token_stride=132) == ALIGN
    assert c(dtype=1, token_stride=136) == c(dtype=1, k_scales=A16 + 2) == c(table=A16 + 1) == c(lengths=A16 + 2) == ALIGN
    if call is not append:
        assert c(Hq=1024, heads=1024, qr=1 << 20, batch=4097) == SHAPE
    for good in (dict(), dict(page_size=1024, cols=1 << 20, table_stride=1 << 20), dict(dtype=1), dict(heads=1),
                 dict(pages=(1 << 31) - 1, page_stride=1 << 40)):
        assert c(**good) == ALIGN, good


def test_append_validation(lib):
    def c(**other):
        return append(lib, **other)

    assert c(K=None) == c(V=None) == c(Q=None) == c(O=None) == c(freqs=None) == NULLPTR
    assert c(freqs=None, Q=None, O=None, Hq=0) == NULLPTR  # rotated needs them
    assert c(axes=A16) == NULLPTR
    assert c(freqs=None, rotated=0, Q=None, O=None, Hq=0, pos=A16, n=1) == NULLPTR
    assert c(Hq=0) == c(Hq=-1) == c(Hq=1025, qr=1 << 20, our=1 << 20) == c(Q=None, O=None) == SHAPE
    assert c(T=0) == c(T=-1) == c(T=(1 << 24) + 1) == c(T=1 << 24, Hq=1024, qr=1 << 20) == SHAPE
    assert c(starts=None) == SHAPE and c(starts=None, T=3, V=A16 + 2) == ALIGN
    assert c(rotated=-16) == c(rotated=144) == c(rotated=24) == c(rotated=0) == SHAPE
    assert c(n=1) == c(pos=A16) == c(pos=A16, n=17) == c(pos=A16, n=-1) == SHAPE
    assert c(kr=64) == c(kh=64) == c(vr=FAR) == c(vh=-128) == c(qr=0) == c(qh=FAR) == c(our=100) == c(oh=100) == SHAPE
    assert c(O=A16, our=4096) == SHAPE  # in place with other strides
    assert c(K=A16 + 2) == c(V=A16 + 8) == c(Q=A16 + 4) == c(O=A16 + 2) == c(kr=516) == c(vh=132) == c(qr=2052) == ALIGN
    assert c(starts=A16 + 2) == c(freqs=A16 + 1) == c(pos=A16 + 2, n=1) == c(pos=A16, axes=A16 + 1, n=3) == ALIGN
    assert b"fp4_kv_append" in lib.fp4_last_error()


@pytest.mark.parametrize("call", [decode, prompt])
def test_attention_validation(lib, call):
    def c(**other):
        return call(lib, **other)

    assert c(Q=None) == c(O=None) == c(ws=None) == NULLPTR
    if call is prompt:
        assert c(starts=None) == NULLPTR
        assert c(T=0) == c(T=(1 << 24) + 1) == c(T=1 << 24, Hq=128, qr=1 << 20) == SHAPE
        assert c(starts=A16 + 2) == ALIGN
    assert c(Hq=0) == c(Hq=-4) == c(Hq=6) == c(Hq=1028, qr=1 << 20) == SHAPE
    assert c(scale=0.0) == c(scale=-1.0) == c(scale=float("nan")) == c(scale=float("inf")) == SHAPE
    assert c(window=-1) == c(sinks=-1) == c(qr=64) == c(qh=FAR) == SHAPE
    need = binding.attention_workspace_bytes(3 if call is decode else 7, 3, 16, 4, 128)
    assert c(n=need - 1) == SHAPE and c(n=need, O=A16 + 8) == ALIGN
    assert c(Q=A16 + 2) == c(qr=2052) == c(qh=132) == c(ws=A16 + 8) == ALIGN
    assert call.__name__.encode() in lib.fp4_last_error()


@pytest.mark.parametrize("T,B,Hq,H,D", [(1, 1, 1, 1, 64), (300, 65, 1024, 1, 256), (8192, 1, 32, 8, 128), (70000, 9, 64, 64, 64)])
def test_workspace_bytes_of_both_sides_agree(lib, T, B, Hq, H, D):
    n = binding.attention_workspace_bytes(T, B, Hq, H, D)

    def call(size):
        return prompt(lib, T=T, Hq=Hq, qr=Hq * D, qh=D, batch=B, heads=H, dim=D, token_stride=D, n=size, O=A16 + 8)
    assert call(n - 1) == SHAPE and call(n) == ALIGN


def test_python_calls_refuse_what_the_kernels_cannot_take():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pages = torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16)
    table, lengths, starts = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.arange(5, dtype=torch.int32)
    for call in (lambda: F.fp4_kv_append(x, x, pages, pages, table, lengths), lambda: F.fp4_kv_append(None, x, pages, pages, table, lengths),
                 lambda: F.fp4_kv_append(x[0], x, pages, pages, table, lengths),
                 lambda: F.fp4_attention_decode(x, pages, pages, table, lengths),
                 lambda: F.fp4_attention_decode(x.float(), pages, pages, table, lengths),
                 lambda: F.fp4_attention_prompt(x, pages, pages, table, lengths, starts),
                 lambda: F.fp4_attention_prompt(x, pages, pages, table, lengths, None)):
        with pytest.raises(ValueError):
            call()
