"""Calls of nothing (no sequence, no row, no head, no dim) are refused as any wrong operand is, by the Python checks; the compiled ones
are asked in test_gpu_attention_refusals.py."""
import pytest
import torch

import microscaling_fp4_quantized_amd as F
from microscaling_fp4_quantized_amd import binding as B


class OnDevice(torch.Tensor):
    """A CPU tensor that the checks take for one on the device; nothing is launched with it."""
    is_cuda = True


def tensors(T=3, nB=3, Hq=4, H=2, D=64, P=5, S=16, cols=2):
    def new(dtype, *shape):
        return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)
    pages = new(torch.bfloat16, P, H, S, D)
    return dict(q=new(torch.bfloat16, T, Hq, D), k_pages=pages, v_pages=pages, table=new(torch.int32, nB, cols),
                lengths=new(torch.int32, nB)), new(torch.int32, nB + 1)


@pytest.fixture(autouse=True)
def _python_checks(monkeypatch):
    monkeypatch.setattr(B, "_FAST", False)

    def launched(*args):
        raise AssertionError("launched")
    monkeypatch.setattr(B, "_enqueue", launched)


def test_what_passes_gets_to_the_launch():
    """So that a refusal below is one of the sizes it names."""
    args, starts = tensors()
    ws = torch.zeros(1 << 25, dtype=torch.uint8).as_subclass(OnDevice)
    for call in (lambda: F.fp4_attention_decode(**args, workspace=ws), lambda: F.fp4_attention_prompt(**args, starts=starts, workspace=ws)):
        with pytest.raises(AssertionError, match="launched"):
            call()


EMPTY = [dict(T=0, nB=0), dict(T=0), dict(H=0), dict(H=0, Hq=0), dict(Hq=0), dict(Hq=1), dict(D=0), dict(nB=0)]


@pytest.mark.parametrize("empty", EMPTY, ids=str)
def test_calls_of_nothing_are_refused(empty):
    args, starts = tensors(**empty)
    out = torch.zeros_like(args["q"])
    ws = torch.zeros(1 << 25, dtype=torch.uint8).as_subclass(OnDevice)
    for more in ({}, dict(out=out, workspace=ws)):
        with pytest.raises(ValueError):
            F.fp4_attention_decode(**args, **more)
        with pytest.raises(ValueError):
            F.fp4_attention_prompt(**args, starts=starts, **more)


@pytest.mark.parametrize("sizes", [(0, 0, 32, 8, 128), (0, 1, 32, 8, 128), (1, 0, 32, 8, 128), (1, 1, 0, 8, 128), (1, 1, 4, 8, 128),
                                   (1, 1, 12, 8, 128), (1, 1, 8, 0, 128), (1, 1, 8, 8, 0), (-1, 1, 8, 8, 64)])
def test_workspace_of_nothing_is_refused(sizes):
    with pytest.raises(ValueError):
        F.attention_workspace_bytes(*sizes)
