"""Compiles csrc/choices.hpp (host code without HIP) with a small main, so that tests can ask it what it chooses."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "microscaling_fp4_quantized_amd", "csrc")


def compile_choices(directory, body):
    """A function: lines of numbers to the numbers that `body` prints, which reads the former with std::scanf."""
    cxx = shutil.which("g++") or shutil.which("c++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    source, program = os.path.join(directory, "choices.cpp"), os.path.join(directory, "choices")
    with open(source, "w") as f:
        f.write(f'#include <cstdio>\n#include "{os.path.join(CSRC, "choices.hpp")}"\nint main() {{\n{body}\nreturn 0;\n}}\n')
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", source, "-o", program], check=True)

    def ask(rows):
        text = "".join(" ".join(map(str, r)) + "\n" for r in rows)
        out = subprocess.run([program], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return ask
