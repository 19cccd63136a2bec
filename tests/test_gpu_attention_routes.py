"""The calls of tests/attention_routes.py, which reach every kernel of the two attentions, against float64, element by element with the
tolerance that paged_plain.attention derives; nothing behind the workspace's bytes is written."""
import pytest
import torch

import attention_routes as R
import microscaling_fp4_quantized_amd as F
from microscaling_fp4_quantized_amd import binding as B
from paged_plain import Cache, attention
from test_gpu_attention import check, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


def run(dim, e4m3, call):
    Hq, H, page, layout, lengths, news, window, sinks, more, gone = call
    c = Cache(lengths, H, dim, page, e4m3, layout, cols_more=more).fill()
    for n, (b, col) in enumerate(gone):
        c.table[b, col] = (-1, c.P, 2 ** 31 - 1)[n % 3]
    args, scale, pad = c.device(), dim ** -0.5, R.PAD if news else 0
    st = [0, *torch.tensor(news or [1] * len(lengths)).cumsum(0).tolist()]
    q = queries(st[-1] + pad, Hq, dim)
    out = torch.full((st[-1] + pad, Hq, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    size = F.attention_workspace_bytes(st[-1] + pad, len(lengths), Hq, H, dim)
    memory = torch.full((size + (8 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    given = dict(window=window, sinks=sinks, out=out, workspace=memory[:size], **c.more)
    if news:
        F.fp4_attention_prompt(q.cuda(), *args, torch.tensor(st, dtype=torch.int32).cuda(), **given)
    else:
        F.fp4_attention_decode(q.cuda(), *args, **given)
    want, tol = attention(c, q[:st[-1]], st, scale, window, sinks, gone)
    check(out[:st[-1]], want, tol, f"{'prompt' if news else 'decode'} D {dim} e4m3 {e4m3} {layout} heads {Hq}/{H}")
    assert (out[st[-1]:] == 7).all() and (memory[size:] == 0xA5).all()


def _flat(routes):
    return [pytest.param(key[0], key[1], call, id="-".join(map(str, key)) + f"-{i}") for key, calls in routes.items() for i, call in enumerate(calls)]


@pytest.mark.parametrize("dim,e4m3,call", _flat(R.PROMPT))
def test_prompt(dim, e4m3, call):
    run(dim, e4m3, call)


@pytest.mark.parametrize("dim,e4m3,call", _flat(R.DECODE))
def test_decode(dim, e4m3, call):
    run(dim, e4m3, call)


@pytest.mark.parametrize("dim,e4m3", sorted(R.DECODE_WIDE))
def test_decode_joined_side_by_side(dim, e4m3):
    run(dim, e4m3, R.DECODE_WIDE[dim, e4m3])
