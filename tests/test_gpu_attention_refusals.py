"""What tests/test_attention_refusals_cpu.py asks of the Python checks, with operands on the GPU and through the compiled checks too."""
import pytest
import torch

import microscaling_fp4_quantized_amd as F
from microscaling_fp4_quantized_amd import binding as B
from test_attention_refusals_cpu import EMPTY

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("empty", EMPTY, ids=str)
def test_calls_of_nothing_are_refused(empty, compiled, monkeypatch):
    if not compiled:
        monkeypatch.setattr(B, "_FAST", False)
    n = dict(T=3, nB=3, Hq=4, H=2, D=64)
    n.update(empty)

    def new(dtype, *shape):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    pages, q = new(torch.bfloat16, 5, n["H"], 16, n["D"]), new(torch.bfloat16, n["T"], n["Hq"], n["D"])
    cache = (pages, pages.clone(), new(torch.int32, n["nB"], 2), new(torch.int32, n["nB"]))
    starts, ws = new(torch.int32, n["nB"] + 1), new(torch.uint8, 1 << 25)
    for more in ({}, dict(out=torch.zeros_like(q), workspace=ws)):
        with pytest.raises((ValueError, F.Fp4Error)):
            F.fp4_attention_decode(q, *cache, **more)
        with pytest.raises((ValueError, F.Fp4Error)):
            F.fp4_attention_prompt(q, *cache, starts, **more)
    torch.cuda.synchronize()


@pytest.mark.parametrize("q", [lambda: torch.zeros((), dtype=torch.bfloat16, device="cuda"),
                               lambda: torch.zeros(3, 4, dtype=torch.bfloat16, device="cuda")])
def test_queries_of_other_dimensions_are_refused(q):
    pages = torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    cache = (pages, pages.clone(), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        F.fp4_attention_decode(q(), *cache, out=torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda"),
                               workspace=torch.zeros(1 << 25, dtype=torch.uint8, device="cuda"))
