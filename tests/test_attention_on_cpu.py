"""The two attentions' own source, compiled for the CPU with a workgroup of fibers (tests/host_gpu): no access leaves its buffer, lanes of
different orders give the same bits (no wave reads what another writes without a barrier between), and sampled rows are float64's.

Every variant of the prompt kernel is forced onto windows, first tokens, ragged rows and tiles past the last one, heads of 64 in four waves
among them; the calls of attention_routes.py go the way that the rule has for them.
"""
import concurrent.futures
import os
import re
import subprocess

import pytest

import attention_routes as R

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "microscaling_fp4_quantized_amd", "csrc")
SOURCES = ("attention_decode.hip", "attention_prompt.hip", "attention_device.hpp", "paged.hpp", "fp8_device.hpp", "operators.hpp", "common.hpp",
           "choices.hpp")


def on_the_cpu(text):
    """What a CPU has no form of: empty asm that holds registers, the bit fields, scalar loads, dynamic LDS."""
    text = re.sub(r'asm volatile\("" : "\+[va]"\([^;]*\)\);', ";", text)
    text = re.sub(r'asm\("v_bfe_i32 .*?\);', "for (int k = 0; k < 4; ++k) off[k] = 0u - (hidden >> (i + k) & 1u);", text, flags=re.S)
    text = text.replace("*(const __attribute__((address_space(4))) int*)(reinterpret_cast<uintptr_t>(p))", "*p")
    text = text.replace("extern __shared__ __align__(16) uint8_t memory[];", "uint8_t* const memory = host::lds;")
    text = text.replace("__shared__ alignas(16)", "alignas(16) static")
    text = text.replace('"../../include/', f'"{os.path.dirname(os.path.dirname(CSRC))}/include/')
    assert "asm" not in re.sub(r"//.*", "", text) and "address_space" not in text
    return text


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    clang = next((c for c in ("/opt/rocm/llvm/bin/clang++", "/opt/rocm/bin/amdclang++") if os.path.exists(c)), None)
    if clang is None:
        pytest.skip("no clang")
    directory = tmp_path_factory.mktemp("attention")
    for name in SOURCES:
        with open(os.path.join(CSRC, name)) as f:
            (directory / name).write_text(on_the_cpu(f.read()))
    out = str(directory / "attention")
    subprocess.run([clang, "-x", "c++", "-O2", "-std=c++17", "-ffp-contract=off", "-w", "-I", os.path.join(HERE, "host_gpu"), "-I", str(directory),
                    os.path.join(HERE, "host_gpu", "attention.cpp"), "-o", out], check=True)
    return out


def run(program, jobs):
    """Each job both with guards behind and, lanes in another order, before its buffers."""
    def one(args):
        got = subprocess.run([program, *map(str, args)], capture_output=True, text=True, timeout=300)
        assert got.returncode == 0, (args, got.stderr)
        return got.stdout.split()
    both = [job(front, order) for job in jobs for front, order in ((0, 0), (1, 7))]
    with concurrent.futures.ThreadPoolExecutor(max_workers=8) as pool:
        results = list(pool.map(one, both))
    for args, a, b in zip(both[::2], results[::2], results[1::2]):
        assert a[0] == b[0] == "1" and float(a[1]) <= 1 and float(b[1]) <= 1, (args, a, b)
        assert a[2] == b[2], args


def job(prompt, waves, splits, dim, e4m3, Hq, H, page, tokens, window, sinks, more, lengths, news, check=12, pad=3):
    def args(front, order):
        return (prompt, waves, splits, dim, int(e4m3), Hq, H, page, int(tokens), window, sinks, more, front, order, check, pad, len(lengths), *lengths,
                *(news if prompt else ()))
    return args


@pytest.mark.parametrize("dim,e4m3,waves,split", sorted(R.PROMPT))
def test_every_prompt_kernel(program, dim, e4m3, waves, split):
    # splits as many as the workspace has room for: 512 / 4 tiles of 128 rows, and no more than 64
    shapes = [(8, 1, 16, True, 100, 4, 1, [450, 33, 300], [300, 33, 1]), (3, 3, 32, False, 0, 0, 2, [90, 260, 64], [90, 7, 0])]
    run(program, [job(1, waves, 3 if split else 1, dim, e4m3, *shape) for shape in shapes])


def test_a_window_over_many_tiles(program):
    """Heads of 64 in bf16 with a window and first tokens: the sizes of a layer, fewer tokens."""
    run(program, [job(1, waves, 1, 64, False, 16, 2, 16, True, 256, 4, 1, [700, 300], [700, 300]) for waves in (4, 8)])


@pytest.mark.parametrize("dim,e4m3,beside,whole", sorted(R.DECODE))
def test_every_decode_kernel(program, dim, e4m3, beside, whole):
    run(program, [job(0, 0, 0, dim, e4m3, Hq, H, page, layout == "tokens", window, sinks, more, lengths, None)
                  for Hq, H, page, layout, lengths, _, window, sinks, more, _ in R.DECODE[dim, e4m3, beside, whole]])
