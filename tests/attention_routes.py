"""Calls of the two attentions by the kernels that they reach on 256 CUs. tests/test_attention_routes_cpu.py checks that they do (choices.hpp
decides), tests/test_gpu_attention_routes.py checks their results against float64.

PROMPT: (dim, 8 bits, waves, split) -> calls; DECODE: (dim, 8 bits, heads side by side of a workgroup, sequences whole) -> calls. A call:
query heads, heads, page size, layout, lengths, new rows (prompt), window, first tokens, columns of the table past the longest sequence,
(sequence, column) of pages that are none. Prompts come with PAD rows of nobody.
"""

PAD = 3

# few rows behind long caches: 512 rows of 16 over 2 heads are 32 tiles of 256 rows, in 8 parts one full round of eight waves. More than one
# sequence, rows that do not fill the last tile of 256, windows with first tokens, missing pages, a row that sees nothing of its first page
_EIGHT_SPLIT = [
    (16, 2, 32, "heads", [2900, 1300], [290, 219], 0, 0, 1, [(0, 3), (1, 0)]),
    (16, 2, 64, "tokens", [2600, 1700, 70], [301, 150, 40], 1500, 70, 40, [(0, 25), (2, 0), (2, 1)]),
    (16, 16, 16, "both", [2900], [493], 0, 0, 1, [(0, 100)]),
]
_FOUR_SPLIT = [
    (8, 2, 32, "gaps", [1500, 40, 333], [3, 1, 60], 0, 0, 1, [(0, 7)]),
    (6, 2, 16, "heads", [2000, 900], [130, 77], 400, 20, 3, [(0, 110), (1, 0)]),
]
_EIGHT_WHOLE = [
    (64, 4, 32, "tokens", [900, 70, 201], [900, 70, 130], 0, 0, 1, [(0, 2)]),
    (64, 64, 16, "heads", [1100], [1029], 333, 17, 0, [(0, 0)]),
]
_FOUR_WHOLE = [
    (4, 2, 64, "both", [200, 33, 256], [150, 33, 7], 0, 0, 0, [(1, 0)]),
    (40, 8, 16, "tokens", [250, 129], [250, 1], 50, 3, 0, [(0, 5)]),
]
PROMPT = {
    (64, False, 4, True): _FOUR_SPLIT, (64, False, 4, False): _FOUR_WHOLE, (64, False, 8, False): _EIGHT_WHOLE,
    (64, True, 4, True): _FOUR_SPLIT, (64, True, 4, False): _FOUR_WHOLE + _EIGHT_WHOLE[:1],
    (128, False, 4, True): _FOUR_SPLIT, (128, False, 4, False): _FOUR_WHOLE, (128, False, 8, True): _EIGHT_SPLIT, (128, False, 8, False): _EIGHT_WHOLE,
    (128, True, 4, True): _FOUR_SPLIT, (128, True, 4, False): _FOUR_WHOLE, (128, True, 8, True): _EIGHT_SPLIT, (128, True, 8, False): _EIGHT_WHOLE,
    (256, False, 4, True): _FOUR_SPLIT, (256, False, 4, False): _FOUR_WHOLE,
    (256, True, 4, True): _FOUR_SPLIT, (256, True, 4, False): _FOUR_WHOLE,
}


def _decode(H, Hq, layout, whole):
    if whole:
        return [(Hq, H, 16, layout, [1, 0, 40, 97, 128], None, 0, 0, 0, [(2, 1)]), (Hq, H, 32, layout, [100, 3], None, 33, 5, 0, [(0, 0)])]
    return [(Hq, H, 16, layout, [2000, 1, 0, 333], None, 0, 0, 9, [(0, 50), (3, 0)]), (Hq, H, 64, layout, [700, 3100], None, 600, 70, 40, [(1, 45)])]


def _beside(beside):
    """Heads and layouts that go one, two or four to a workgroup."""
    return {1: (3, 6, "heads"), 2: (6, 12, "tokens"), 4: (4, 72, "tokens")}[beside]


DECODE = {(dim, e4m3, beside, whole): _decode(*_beside(beside), whole)
          for dim, e4m3, most in ((64, False, 4), (64, True, 4), (128, False, 2), (128, True, 4), (256, False, 1), (256, True, 2))
          for beside in (1, 2, 4) if beside <= most for whole in (False, True)}
# a join whose workgroups have several heads: batches of many rows
DECODE_WIDE = {(dim, e4m3): (32, 8, 16, "heads", [(37 * i) % 1300 for i in range(33)], None, 0, 0, 1, [(5, 3)])
               for dim in (64, 128, 256) for e4m3 in (False, True)}
