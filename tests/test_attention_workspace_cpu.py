"""The attention calls' workspace: what include/fp4.h and the Python function say is the same, grows with rows and sequences (so that one
sized for a program's longest call serves every other), and holds whatever a call may put there."""
import os
import random
import shutil
import subprocess

import pytest

import microscaling_fp4_quantized_amd as F

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADS = [(1, 1), (8, 8), (32, 8), (64, 8), (64, 64), (16, 4), (64, 1), (12, 12), (7, 7), (1024, 1), (1024, 1024), (40, 1), (66, 2)]
ROWS = sorted({max(1, n + d) for n in (1, 2, 64, 100, 512, 1024, 2048, 4096, 8192, 16384, 65536, 1 << 20) for d in (-1, 0, 1)})


@pytest.mark.parametrize("Hq,H", HEADS)
def test_bytes_grow_with_rows_and_sequences(Hq, H):
    for B in (1, 2, 9, 64, 300, 4096):
        sizes = [F.attention_workspace_bytes(T, B, Hq, H, 128) for T in ROWS]
        assert sizes == sorted(sizes), B
    for T in ROWS:
        sizes = [F.attention_workspace_bytes(T, B, Hq, H, 128) for B in range(1, 700)]
        assert sizes == sorted(sizes), T


def test_the_header_agrees_and_every_part_has_its_place(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    source, program = tmp_path / "bytes.cpp", tmp_path / "bytes"
    source.write_text(f'#include <cstdio>\n#include <cstdint>\n#include "{ROOT}/include/fp4.h"\n' + """
int main() {
  long long T, B, q, h, d;
  while (std::scanf("%lld %lld %lld %lld %lld", &T, &B, &q, &h, &d) == 5)
    std::printf("%zu %lld %lld\\n", FP4_ATTENTION_WORKSPACE_BYTES(T, B, q, h, d), (long long)FP4_ATTENTION_SPLITS(T, B, q, h),
                (long long)FP4_ATTENTION_PIECES(B, FP4_ATTENTION_UNITS_(q, h)));
}""")
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", str(source), "-o", str(program)], check=True)
    rng = random.Random(1)
    cases = [(T, B, *heads, 64) for T in ROWS for B in (1, 2, 9, 300) for heads in HEADS]
    cases += [(rng.randint(1, 5000), rng.randint(1, 400), *rng.choice(HEADS), rng.choice([64, 128, 256])) for _ in range(20000)]
    text = "".join(" ".join(map(str, c)) + "\n" for c in cases)
    out = subprocess.run([str(program)], input=text, capture_output=True, text=True, check=True).stdout
    for case, line in zip(cases, out.splitlines()):
        T, B, Hq, H, D = case
        size, splits, pieces = map(int, line.split())
        assert size == F.attention_workspace_bytes(*case), case
        per = Hq * (D + 2) * 4  # a partial result of every query head
        assert (splits == 1 or splits * T * per <= size) and (pieces + B) * per <= size, case
