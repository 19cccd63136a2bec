"""A wait for LDS DMA that leaves the youngest N loads in flight is right only if N loads were really issued after the one it
waits for. DMA loads are (each is a side effect of its own); loads to registers need not be, because the compiler may merge
or drop them. So the counts in the kernels' sources are made of numbers of DMA loads only.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "microscaling_fp4_quantized_amd", "csrc")

# what a count may name: DMA loads of a stage, block or fetch, and how many of those are ahead
DMA = {"moe.hip": {"kDma"}, "gemm_fp8_split.hip": {"SLOTS", "C", "LOADS"}, "gemm_fp8_ring.hip": {"D", "KB", "A_WL", "B_WL"}}


@pytest.mark.parametrize("name", sorted(DMA))
def test_counted_waits_count_dma_only(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    counts = re.findall(r"\bwait_vmcnt<([^;]*?)>\(\);", text)
    assert counts
    for c in counts:
        assert set(re.findall(r"[A-Za-z_]\w*", c)) <= DMA[name], c


def test_the_experts_dma_loads_are_counted_as_issued():
    """kDma against the DMA instructions of a fetch: two pieces of eight rows for each tile of sixteen."""
    with open(os.path.join(CSRC, "moe.hip")) as f:
        text = f.read()
    assert re.findall(r"constexpr int kDma = ([^;]*);", text) == ["2 * kTiles"] * 2
    fetches = re.findall(r"auto fetch = \[&\].*?\n  };", text, re.S)
    assert len(fetches) == 2
    for f in fetches:
        assert f.count("load_lds(") == 1
        loops = re.findall(r"for \(int (\w) = 0; \1 < (\w+); \+\+\1\)", f[:f.index("load_lds(")])
        assert loops[-2:] == [("t", "kTiles"), ("q", "2")]
