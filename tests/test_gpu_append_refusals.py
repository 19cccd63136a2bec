"""Positions of no axis are refused by the compiled and by the Python checks, and nothing is written."""
import pytest
import torch

import microscaling_fp4_quantized_amd as F
from microscaling_fp4_quantized_amd import binding as B
from test_append_refusals_cpu import operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("compiled", [True, False])
def test_positions_of_no_axis_are_refused(compiled, monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not compiled:
        monkeypatch.setattr(B, "_FAST", False)

    def new(dtype, *shape):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    args, more = operands(new, (0,))
    args[0].fill_(1)
    args[5].fill_(1)
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7)
    for given in ({}, dict(q=q, out=out)):
        with pytest.raises(ValueError):
            F.fp4_kv_append(*args, **more, **given)
    torch.cuda.synchronize()
    assert (args[2] == 0).all() and (out == 7).all()
