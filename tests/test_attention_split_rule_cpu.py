"""How many waves share a tile where prompt attention splits a row's tokens (csrc/choices.hpp): by the workgroups that there are, not at
single sizes."""
import pytest

from attention_choices import prompt_choice

EIGHT = [  # T, batch, query heads, heads: one full round of workgroups of 256 rows, in at most 8 parts
    *((T, 2, 32, 8) for T in (961, 1000, 1023, 1024, 449, 500, 512, 230, 256)),
    *((T, 1, 16, 16) for T in (400, 512, 769, 900, 1024, 1793, 2000, 2048)), (256, 3, 64, 8), (512, 3, 64, 8),
]
FOUR = [  # too many parts, CUs that would idle, or a second round
    *((T, 2, 32, 8) for T in (97, 128, 193, 200, 520, 641, 680, 900, 960, 1)), *((T, 1, 16, 16) for T in (130, 256, 300, 600, 768, 1025, 1200, 1280)),
    (1024, 32, 32, 8),  # 32 sequences of 32 tokens: tiles half empty
]


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    return prompt_choice(str(tmp_path_factory.mktemp("prompt")))


@pytest.mark.parametrize("e4m3", [0, 1])
def test_eight_waves_with_a_split(choice, e4m3):
    calls = [(128, e4m3, *c, 16384, 0, 0) for c in EIGHT + FOUR]
    for call, (waves, splits, wide) in zip(calls, choice(calls)):
        assert splits > 1 and wide > 0, call
        assert waves == (8 if call[2:6] in EIGHT else 4), call


def test_heads_of_64_and_256_take_four_with_a_split(choice):
    for dim, e4m3 in ((64, 0), (64, 1), (256, 0), (256, 1)):
        for waves, splits, _ in choice([(dim, e4m3, *c, 16384, 0, 0) for c in EIGHT]):
            assert waves == 4 and splits > 1


def test_a_row_more_or_less_changes_no_more_than_one_step(choice):
    """Within a number of parts, eight waves are taken over a range of rows that ends with the last tile's last row."""
    calls = [(128, 0, T, 2, 32, 8, 16384, 0, 0) for T in range(1, 1025)]
    got = choice(calls)
    ranges = []
    for (_, _, T, *_), (waves, splits, _) in zip(calls, got):
        if waves == 8:
            if ranges and ranges[-1][1] == T - 1:
                ranges[-1][1] = T
            else:
                ranges.append([T, T])
    assert ranges and all(last - first >= 31 and last * 4 % 256 == 0 for first, last in ranges), ranges
