"""Every kernel of the two attentions that the choice can take is there in tests/attention_routes.py, and its calls take it."""
import itertools

import pytest

import attention_routes as R
from attention_choices import decode_choice, prompt_choice


@pytest.fixture(scope="module")
def prompt(tmp_path_factory):
    return prompt_choice(str(tmp_path_factory.mktemp("prompt")))


@pytest.fixture(scope="module")
def decode(tmp_path_factory):
    return decode_choice(str(tmp_path_factory.mktemp("decode")))


def room(call):
    _, _, page, _, lengths, _, _, _, more, _ = call
    return page * max(max(-(-n // page) for n in lengths) + more, 1)


def test_prompts_take_the_kernels_they_are_there_for(prompt):
    for (dim, e4m3, waves, split), calls in R.PROMPT.items():
        for call in calls:
            Hq, H, _, _, lengths, news, window, sinks, _, gone = call
            (got,) = prompt([(dim, int(e4m3), sum(news) + R.PAD, len(news), Hq, H, room(call), window, sinks)])
            assert (got[0], got[1] > 1) == (waves, split), (dim, e4m3, call, got)
            assert gone and all(m <= n for m, n in zip(news, lengths))


def test_every_prompt_kernel_that_a_call_can_take_is_listed(prompt):
    calls = [(dim, e4m3, T, B, Hq, H, room, window, 4) for dim, e4m3 in itertools.product((64, 128, 256), (0, 1))
             for T in (1, 16, 100, 128, 256, 400, 500, 512, 700, 1000, 1024, 2000, 2048, 4096, 20000) for B in (1, 2, 9, 64) if T >= B
             for Hq, H in ((1, 1), (8, 1), (16, 2), (16, 16), (32, 8), (64, 8), (64, 64)) for room in (64, 300, 2048, 32768) for window in (0, 1000)]
    reached = {(c[0], bool(c[1]), waves, splits > 1) for c, (waves, splits, _) in zip(calls, prompt(calls))}
    assert reached == set(R.PROMPT)


def test_decodes_take_the_kernels_they_are_there_for(decode):
    for (dim, e4m3, beside, whole), calls in R.DECODE.items():
        for call in calls:
            Hq, H, _, layout, lengths, _, window, sinks, _, _ = call
            (got,) = decode([(dim, int(e4m3), len(lengths), Hq, H, room(call), window, sinks, int(layout == "tokens"))])
            assert got[:2] == (beside, whole) and (got[3] > 0) == (not whole), (dim, e4m3, call, got)
    for (dim, e4m3), call in R.DECODE_WIDE.items():
        Hq, H, _, layout, lengths, _, window, sinks, _, _ = call
        (got,) = decode([(dim, int(e4m3), len(lengths), Hq, H, room(call), window, sinks, 0)])
        assert got[3] == 1024 // dim and not got[1], (dim, e4m3, got)


def test_every_decode_kernel_that_a_call_can_take_is_listed(decode):
    calls = [(dim, e4m3, B, Hq, H, room, window, 4, beside) for dim, e4m3 in itertools.product((64, 128, 256), (0, 1))
             for B in (1, 3, 64, 300) for Hq, H in ((1, 1), (6, 2), (12, 12), (32, 8), (64, 1), (9, 3)) for room in (64, 400, 2000, 131072)
             for window in (0, 100) for beside in (0, 1)]
    reached = {(c[0], bool(c[1]), beside, bool(whole)) for c, (beside, whole, _, _) in zip(calls, decode(calls))}
    assert reached == set(R.DECODE)
