"""The summaries of perf/time_operators.py on small tables as rocprofv3 writes them."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def tool():
    spec = importlib.util.spec_from_file_location("time_operators", os.path.join(ROOT, "perf", "time_operators.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_trace(tool, tmp_path, capsys):
    head = "Kernel_Name,Grid_Size_X,Grid_Size_Y,Grid_Size_Z,Workgroup_Size_X,LDS_Block_Size,VGPR_Count,Scratch_Size,Start_Timestamp,End_Timestamp"
    name = "\"void fp4::(anonymous namespace)::gemm<1, 2>(int, int)\""
    rows = [f"{name},512,2,4,256,0,28,0,{s},{e}" for s, e in ((0, 3000), (10000, 12000), (20000, 26000))]
    path = tmp_path / "t.csv"
    path.write_text("\n".join([head, *rows, "library_kernel,1,1,1,1,0,1,0,0,9000"]) + "\n")
    tool.trace(str(path))
    lines = capsys.readouterr().out.splitlines()
    assert len(lines) == 2 and lines[1].startswith("gemm<1, 2> ")
    assert lines[1].split()[2:] == ["4096", "256", "0", "28", "0", "3", "3.00", "2.00"]


def test_counters(tool, tmp_path, capsys):
    path = tmp_path / "c.csv"
    path.write_text("Kernel_Name,Grid_Size,Counter_Name,Counter_Value\n" + "".join(
        f"void fp4::(anonymous namespace)::{k}(int),64,SQ_WAVES,{v}\n" for k, v in (("a", 1), ("a", 3), ("b", 100))))
    tool.counters(str(path), "a")
    lines = [line.split() for line in capsys.readouterr().out.splitlines()]
    assert [line[0] for line in lines] == ["a"]
    assert lines[0][1:4] == ["64", "SQ_WAVES", "2"] and lines[0][-2:] == ["2", "dispatches"]
