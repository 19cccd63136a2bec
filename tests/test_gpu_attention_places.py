"""Places at the ends of what a cache may be: tokens that the table has no room for, with paged_plain's element by element tolerance, and
scales that lie past 2^31 elements and 2^32 bytes."""
import pytest
import torch

import microscaling_fp4_quantized_amd as F
from microscaling_fp4_quantized_amd import binding as B
from paged_plain import Cache, attention
from parity import say
from test_gpu_attention import check, queries
from test_gpu_attention_calls import bits, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


@pytest.mark.parametrize("D,e4m3", [(64, False), (128, True), (256, False)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (10, 0), (10, 3), (100, 0)])
def test_lengths_past_the_table(D, e4m3, window, sinks):
    """70 tokens where the table has room for 64: the last six are as of no page, the rows' places count all 70."""
    c = Cache([64], 2, D, 16, e4m3, cols_more=0).fill()
    args = c.device()
    args[3].fill_(70)
    # the same for the reference: a fifth column that is no page
    c.lengths, gone = torch.tensor([70], dtype=torch.int32), [(0, 4)]
    c.keys[0], c.values[0] = (torch.cat([x, torch.zeros(6, 2, D, dtype=torch.float64)]) for x in (c.keys[0], c.values[0]))
    q, scale = queries(20, 4, D), D ** -0.5
    want, tol = attention(c, q[:1], [0, 1], scale, window, sinks, gone)
    check(F.fp4_attention_decode(q[:1].cuda(), *args, window=window, sinks=sinks, **c.more), want, tol, "decode past the table")
    want, tol = attention(c, q, [0, 20], scale, window, sinks, gone)
    got = F.fp4_attention_prompt(q.cuda(), *args, torch.tensor([0, 20], dtype=torch.int32).cuda(), window=window, sinks=sinks, **c.more)
    check(got, want, tol, "prompt past the table")


def test_scales_past_2_31_elements():
    """Pages of scales 2^28 elements apart: written and read as those that lie together."""
    H, S, D, P = 4, 32, 128, 10
    say("scales past 2^31")
    lengths = torch.tensor([200, 64], dtype=torch.int32, device="cuda")
    table = torch.tensor([[9, 8, 0, 5, 7, 1, 2], [4, 3, -1, -1, -1, -1, -1]], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 200, 264], dtype=torch.int32, device="cuda")
    x = normal(3, 264, 16 + 2 * H, D)
    step = (1 << 28) + 2 * H * S
    far = torch.empty((P - 1) * step + 2 * H * S, dtype=torch.float32, device="cuda")
    assert (P - 1) * step > 1 << 31
    got = []
    for sk, sv in ((far.as_strided((P, H, S), (step, S, 1), 0), far.as_strided((P, H, S), (step, S, 1), H * S)),
                   [torch.empty(P, H, S, device="cuda") for _ in range(2)]):
        k, v = (torch.zeros(P, H, S, D, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
        more = dict(k_scales=sk, v_scales=sv)
        sk.fill_(0)
        sv.fill_(0)
        q = x[:, :16]
        F.fp4_kv_append(x[:, 16:16 + H], x[:, 16 + H:], k, v, table, lengths, starts, **more)
        got.append([F.fp4_attention_prompt(q, k, v, table, lengths, starts, **more), F.fp4_attention_decode(q[:2], k, v, table, lengths, **more),
                    sk.clone(), sv.clone(), k, v])
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(bits(a), bits(b))
    assert all(t.isfinite().all() and t.any() for t in got[0][:4])
    del far
    torch.cuda.empty_cache()
