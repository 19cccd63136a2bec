"""Launches of more work-items than one grid dimension holds (HIP: below 2^32)."""
import pytest

from host_program import compile_choices


@pytest.fixture(scope="module")
def grid(tmp_path_factory):
    return compile_choices(str(tmp_path_factory.mktemp("grid")), """
  long long n; int t;
  while (std::scanf("%lld %d", &n, &t) == 2) {
    const fp4::Grid g = fp4::grid_of(n, t);
    std::printf("%u %u\\n", g.x, g.y);
  }""")


def test_grids_hold_every_workgroup_once_and_stay_below_the_limit(grid):
    sizes = [1, 7, 8, 1 << 20, (1 << 22) - 1, 1 << 22, (1 << 23) - 1, 1 << 23, (1 << 24) - 1, 1 << 24, (1 << 24) + 1, 1 << 25,
             (1 << 25) + 12345, 1 << 27, (1 << 31) - 1]
    rows = [(n, t) for n in sizes for t in (64, 256, 512, 1024)]
    for (n, t), (x, y) in zip(rows, grid(rows)):
        assert x * t < 1 << 32 and y < 1 << 16, (n, t)
        assert x * y >= n > x * (y - 1), (n, t)
        assert y == 1 or x % 8 == 0
        assert y > 1 or x == n
