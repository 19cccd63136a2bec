"""fp4_kv_append's Python checks: positions of no axis are refused. A tensor of nothing has a null pointer, which the library takes for
positions that were not given: the tokens' places were used in silence. The compiled checks are asked in test_gpu_append_refusals.py."""
import pytest
import torch

import microscaling_fp4_quantized_amd as F
from test_attention_refusals_cpu import OnDevice, _python_checks  # noqa: F401


def operands(new, axes):
    k = new(torch.bfloat16, 3, 2, 64)
    pages = new(torch.bfloat16, 5, 2, 16, 64)
    more = {} if axes is None else dict(positions=new(torch.int32, *axes, 3))
    return (k, new(torch.bfloat16, 3, 2, 64), pages, new(torch.bfloat16, 5, 2, 16, 64), new(torch.int32, 3, 2), new(torch.int32, 3)), \
        dict(freqs=new(torch.float32, 32), **more)


def test_positions_of_no_axis_are_refused():
    def new(dtype, *shape):
        return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)
    for axes in (None, (), (1,), (3,)):
        args, more = operands(new, axes)
        with pytest.raises(AssertionError, match="launched"):
            F.fp4_kv_append(*args, **more)
    args, more = operands(new, (0,))
    with pytest.raises(ValueError):
        F.fp4_kv_append(*args, **more)
    with pytest.raises(ValueError):
        F.fp4_kv_append(*args, axes=new(torch.int32, 32), **more)
