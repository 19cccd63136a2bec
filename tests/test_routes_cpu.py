"""Which kernel a call takes (csrc/choices.hpp, compiled alone): every one of them is reached by the calls that the GPU tests
check, and those of tests/operator_routes.py take the ones that they are there for."""
import pytest

import operator_routes as R
import test_gpu_fp8
import test_gpu_moe
from host_program import compile_choices

CUS = 256
WINDOW = 4096  # elements of a row whose scales LDS holds at once


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    return compile_choices(str(tmp_path_factory.mktemp("shape")), f"""
  long long M, N, K;
  while (std::scanf("%lld %lld %lld", &M, &N, &K) == 3) std::printf("%d\\n", fp4::best_shape(M, N, K, {CUS}));""")


@pytest.fixture(scope="module")
def experts(tmp_path_factory):
    """T, k, E, D, I -> two launches?, waves of up and of down in the five."""
    return compile_choices(str(tmp_path_factory.mktemp("experts")), """
  long long T, k, E, D, I;
  while (std::scanf("%lld %lld %lld %lld %lld", &T, &k, &E, &D, &I) == 5) {
    const long long slots = std::min(T * k, E);
    std::printf("%d %d %d\\n", fp4::few_pairs((int)T, (int)k, E, D, I), fp4::expert_waves(D, slots * I / 32),
                fp4::expert_waves(I, slots * D / 64));
  }""")


def test_products_take_the_shapes_they_are_there_for(shape):
    for want, cases in {**R.LINEAR, **{s: R.LINEAR.get(s, []) + [c] for s, c in R.EDGES.items()}}.items():
        for case, (got,) in zip(cases, shape(cases)):
            assert got == want, case


def test_every_ring_refills_its_buffers_and_passes_64_blocks(shape):
    for want, cases in R.LINEAR.items():
        blocks = [K // 128 for _, _, K in cases]
        assert any(b > 8 and b % 2 for b in blocks) and max(blocks) > 64, want
        assert all(N % 2 for _, N, _ in cases)


def test_every_shape_is_checked_against_float64(shape):
    cases = test_gpu_fp8.LINEAR + test_gpu_fp8.SPLIT
    assert {s for s, in shape(cases)} == set(range(8))


def test_experts_take_the_waves_they_are_there_for(experts):
    for case, (few, up, down) in zip(R.EXPERTS, experts([c[:5] for c in R.EXPERTS])):
        T, k, E, D, I, _, want_up, want_down, loads = case
        assert (few, up, down) == (0, want_up, want_down), case
        assert sum(loads) <= T * k and len(loads) <= E
    # several windows with every number of waves that such rows can have, in both products
    assert {c[6] for c in R.EXPERTS if c[3] > WINDOW} == {2, 8}
    assert {c[7] for c in R.EXPERTS if c[4] > WINDOW} == {2, 8}
    # one to four fragments in a pass, and more than one pass, for every number of waves
    for at in (6, 7):
        for waves in (1, 2, 8):
            loads = [n for c in R.EXPERTS if c[at] == waves for n in c[8]]
            assert {-(-min(n, 16) // 4) for n in loads} == {1, 2, 3, 4} and max(loads) > 16, (at, waves)


def test_the_experts_tests_reach_both_forms(experts):
    """SORTED is there for the five launches, and the small cases for the two."""
    ways = experts([(T, k, E, D, I) for T, E, D, I, k, _ in test_gpu_moe.SORTED])
    assert not any(few for few, _, _ in ways)
    assert {up for _, up, _ in ways} == {down for _, _, down in ways} == {1, 2, 8}
    assert any(few for few, _, _ in experts([(T, k, E, D, I) for T, E, D, I, k, _ in test_gpu_moe.EXPERTS]))
