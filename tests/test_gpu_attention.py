"""fp4_attention_decode and fp4_attention_prompt against float64 on the CPU, element by element, with the tolerance that
paged_plain.attention derives. Places that no token holds are NaN in every cache here."""
import pytest
import torch

import microscaling_fp4_quantized_amd as F
from microscaling_fp4_quantized_amd import binding as B
from paged_plain import Cache, attention
from parity import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


def queries(T, Hq, D, seed=2, scale=1.0):
    """Rows in a wider buffer, heads apart."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, Hq + 1, D + 8, generator=g) * scale).bfloat16()[:, :Hq, :D]


def check(got, want, tol, label):
    got = got.cpu().double()
    worst = float(((got - want).abs() / tol.clamp_min(1e-30)).nan_to_num(1e30).max()) if got.numel() else 0.0
    say(f"{label}: {worst:.3f} of the tolerance")
    assert got.isfinite().all() and worst <= 1.0


def run(c, Hq, news=None, scale=None, window=0, sinks=0, pad=0, gone=(), seed=2, qscale=1.0):
    """Decode (news None) or prompt on cache c."""
    D, nB = c.D, len(c.lengths)
    scale = D ** -0.5 if scale is None else scale
    args = c.device()
    label = f"D {D} e4m3 {c.e4m3} {c.layout} page {c.S} heads {Hq}/{c.H} window {window} sinks {sinks}"
    if news is None:
        q = queries(nB, Hq, D, seed, qscale)
        got = F.fp4_attention_decode(q.cuda(), *args, scale=scale, window=window, sinks=sinks, **c.more)
        want, tol = attention(c, q, range(nB + 1), scale, window, sinks, gone)
        return check(got, want, tol, "decode " + label)
    st = [0, *torch.tensor(news).cumsum(0).tolist()]
    q = queries(st[-1] + pad, Hq, D, seed, qscale)
    out = torch.full((st[-1] + pad, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got = F.fp4_attention_prompt(q.cuda(), *args, torch.tensor(st, dtype=torch.int32).cuda(), scale=scale, window=window, sinks=sinks,
                                 out=out, **c.more)
    assert got is out and (out[st[-1]:] == 7).all()
    want, tol = attention(c, q[:st[-1]], st, scale, window, sinks, gone)
    check(got[:st[-1]], want, tol, "prompt " + label)


LAYOUTS = ["heads", "tokens", "both", "gaps"]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_decode_lengths(D, e4m3, layout):
    """One token to many, ends on both sides of a granule, a tile, a page and a piece, none at all."""
    run(Cache([1, 2, 15, 16, 17, 31, 32, 33, 0, 64, 127, 128, 129, 300, 1025], 2, D, 16, e4m3, layout).fill(), 4)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_prompt_lengths(D, e4m3, layout):
    news = [1, 0, 31, 64, 65, 129, 7, 2]
    run(Cache([n + x for n, x in zip(news, (0, 3, 0, 5, 64, 0, 200, 1000))], 2, D, 16, e4m3, layout).fill(), 4, news, pad=3)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 512, 1024])
def test_page_sizes(page):
    c = Cache([700, 5, 1500], 2, 64, page).fill()
    run(c, 4)
    run(c, 4, [300, 5, 70])


@pytest.mark.parametrize("Hq,H", [(1, 1), (7, 7), (3, 1), (10, 2), (16, 1), (17, 1), (48, 1), (40, 1), (64, 2), (130, 1)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_heads(Hq, H, e4m3):
    c = Cache([200, 33], H, 64, 32, e4m3, "both").fill()
    run(c, Hq)
    run(c, Hq, [50, 33])


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 4), (100, 16), (100, 17), (128, 500), (300, 40), (1 << 40, 7)])
@pytest.mark.parametrize("D,e4m3", [(64, False), (128, True), (256, False)])
def test_windows(window, sinks, D, e4m3):
    c = Cache([1, 16, 90, 101, 117, 250, 613, 1300], 2, D, 16, e4m3).fill()
    run(c, 4, window=window, sinks=sinks)
    run(c, 4, [1, 16, 40, 101, 1, 130, 300, 64], window=window, sinks=sinks)


@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_that_are_none(e4m3):
    """Rows whose pages are all missing get zeros; a missing page inside takes its tokens away."""
    c = Cache([100, 40, 333, 20], 2, 64, 16, e4m3).fill()
    gone = [(0, 0), (0, 3), (1, 0), (1, 1), (1, 2), (2, 20), (3, 1)]
    for n, (b, col) in enumerate(gone):
        c.table[b, col] = (-1, c.P, -2 ** 31, 2 ** 31 - 1)[n % 4]
    run(c, 4, gone=gone)
    run(c, 4, [60, 40, 200, 20], gone=gone)
    run(c, 4, [60, 40, 200, 20], window=30, sinks=3, gone=gone)


def test_rows_without_tokens():
    """Lengths of zero and below, and rows that stand before their sequence."""
    c = Cache([5, 9, 40], 1, 64, 16).fill()
    q = queries(3, 2, 64).cuda()
    args = c.device()
    args[3].copy_(torch.tensor([0, -7, 40]))
    got = F.fp4_attention_decode(q, *args)
    assert (got[:2] == 0).all() and got[2].abs().sum() > 0
    args[3].copy_(torch.tensor([3, 0, 40]))
    st = torch.tensor([0, 10, 20, 60], dtype=torch.int32).cuda()
    q = queries(60, 2, 64)
    got = F.fp4_attention_prompt(q.cuda(), *args, st)
    assert (got[:7] == 0).all() and (got[10:20] == 0).all()
    c.lengths = torch.tensor([3, 0, 40], dtype=torch.int32)
    c.keys[0], c.values[0], c.keys[1], c.values[1] = c.keys[0][:3], c.values[0][:3], c.keys[1][:0], c.values[1][:0]
    want, tol = attention(c, q[7:], [0, 3, 3, 43], 0.125)
    rows = torch.cat([torch.arange(7, 10), torch.arange(20, 60)])
    want, tol = attention(c, q[rows], [0, 3, 3, 43], 0.125)
    check(got.cpu()[rows], want, tol, "rows behind those without tokens")


def test_lengths_past_the_table():
    """Tokens that the table has no room for are as of no page; the row's place still counts for its window."""
    c = Cache([64], 1, 64, 16, cols_more=0).fill()
    args = c.device()
    q = queries(1, 2, 64)
    args[3].fill_(70)
    got = F.fp4_attention_decode(q.cuda(), *args)
    want, tol = attention(c, q, range(2), 0.125)
    check(got, want, tol, "length past the table")
    got = F.fp4_attention_decode(q.cuda(), *args, window=10)
    c.keys[0][:60] = -1e4 * q[0, 0].double().sign()  # the reference's way to leave them out: tokens 60..63 are in the window
    k, v = Cache([64], 1, 64, 16, cols_more=0).fill(), None
    z = torch.einsum("hd,jd->hj", q[0].double(), k.keys[0][60:, 0]) * 0.125
    want = torch.softmax(z, 1) @ k.values[0][60:, 0]
    assert (got[0].cpu().double() - want).abs().max() <= 2.0 ** -7 * k.values[0].abs().max()
    args[3].fill_(2 ** 31 - 1)
    got = F.fp4_attention_decode(q.cuda(), *args, window=10)
    assert (got == 0).all()


@pytest.mark.parametrize("qscale", [0.0, 30.0])
def test_flat_and_steep_scores(qscale):
    """All scores equal, and scores hundreds apart, where p under- and the maximum overtakes itself."""
    for e4m3 in (False, True):
        c = Cache([500, 1000], 2, 128, 32, e4m3).fill()
        run(c, 8, qscale=qscale)
        run(c, 8, [300, 100], qscale=qscale)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rising_scores(D):
    """Keys that grow along the sequence: the running maximum moves at every tile."""
    c = Cache([900], 1, D, 16).fill()
    i = torch.arange(900)
    k = c.keys[0] * (i[:, None, None] / 100.0)
    k = k.bfloat16()
    c.k[c.table[0].long()[i // 16], :, i % 16] = k
    c.keys[0] = k.double()
    run(c, 4)
    run(c, 4, [900])


@pytest.mark.parametrize("e4m3", [False, True])
def test_non_finite_values_stay_with_the_rows_that_see_them(e4m3):
    """A NaN in a value or key of one head in the middle of a prompt: rows before it, rows whose window has left it and the other head
    are as without it, rows that see it are no numbers."""
    n, at = 200, 70
    for what in ("value", "key", "infinite value"):
        for window in (0, 50):
            c = Cache([n], 2, 64, 16, e4m3).fill()
            q = queries(n, 4, 64)
            want, tol = attention(c, q, [0, n], 0.125, window)
            p, o = c.place(0, at)
            pages, scales = (c.k, c.ks) if what == "key" else (c.v, c.vs)
            if e4m3 and what == "infinite value":
                scales[p, 0, o] = float("inf")
            elif e4m3:
                pages[p, 0, o, 3] = 0x7F
            else:
                pages[p, 0, o, 3] = float("inf" if what == "infinite value" else "nan")
            args = c.device()
            got = F.fp4_attention_prompt(q.cuda(), *args, torch.tensor([0, n], dtype=torch.int32).cuda(), window=window, **c.more).cpu()
            sees = torch.zeros(n, dtype=torch.bool)
            sees[at:at + (window or n)] = True
            check(got[~sees], want[~sees], tol[~sees], f"rows that do not see the {what}")
            check(got[:, 2:], want[:, 2:], tol[:, 2:], "the other head")
            bad = ~got[sees][:, :2].isfinite()
            assert bad.any(-1).all(), what
            args[3].fill_(at + 20)
            one = F.fp4_attention_decode(q[:1].cuda(), *args, window=window, **c.more)
            assert (~one[0, :2].isfinite()).any(-1).all() and one[0, 2:].isfinite().all()
            args[3].fill_(at + 60)
            one = F.fp4_attention_decode(q[:1].cuda(), *args, window=window, **c.more)
            assert bool(one.isfinite().all()) == bool(window)
    # a NaN in a query is its own row's and head's
    c = Cache([n], 2, 64, 16, e4m3).fill()
    q = queries(n, 4, 64)
    want, tol = attention(c, q, [0, n], 0.125)
    qd = q.cuda()
    qd[90, 1, 7] = float("nan")
    got = F.fp4_attention_prompt(qd, *c.device(), torch.tensor([0, n], dtype=torch.int32).cuda(), **c.more).cpu()
    assert got[90, 1].isnan().all()
    got[90, 1], want[90, 1] = 0, 0
    check(got, want, tol, "the other rows")


def test_many_sequences():
    """More than a wave's lanes."""
    lengths = [(7 * i) % 90 for i in range(150)]
    c = Cache(lengths, 1, 64, 16).fill()
    run(c, 3)
    run(c, 3, [min(n, i % 5) for i, n in enumerate(lengths)], pad=4)


@pytest.mark.parametrize("layout", ["tokens", "gaps", "heads"])
@pytest.mark.parametrize("H,Hq", [(4, 4), (4, 72), (2, 6), (8, 32), (6, 12), (3, 3)])
@pytest.mark.parametrize("D,e4m3", [(64, False), (64, True), (128, False), (128, True), (256, True)])
def test_heads_side_by_side(layout, H, Hq, D, e4m3):
    """Rows of heads that lie next to each other go to one workgroup, two or four at a time; those that do not, one by one."""
    c = Cache([1, 40, 31, 700, 0, 333], H, D, 16, e4m3, layout).fill()
    run(c, Hq)
    run(c, Hq, window=100, sinks=5)


@pytest.mark.parametrize("H,Hq,nB,layout", [(12, 12, 169, "heads"), (24, 24, 85, "tokens"), (24, 48, 85, "heads"), (20, 20, 101, "tokens")])
def test_a_workspace_of_just_its_bytes_is_enough(H, Hq, nB, layout):
    """Where the pieces of a batch, rounded up to whole rounds of workgroups, come to more than the workspace is for."""
    D = 64
    c = Cache([97 + (37 * b) % 120 for b in range(nB)], H, D, 16, False, layout).fill()
    args, q = c.device(), queries(nB, Hq, D)
    bytes_ = F.attention_workspace_bytes(nB, nB, Hq, H, D)
    memory = torch.full((bytes_ + (8 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    got = F.fp4_attention_decode(q.cuda(), *args, workspace=memory[:bytes_], **c.more)
    want, tol = attention(c, q, range(nB + 1), D ** -0.5)
    check(got, want, tol, f"decode {nB} sequences heads {Hq}/{H} {layout}")
    assert (memory[bytes_:] == 0xA5).all()


@pytest.mark.parametrize("H,Hq,news,D,e4m3", [(2, 8, [3, 17], 64, False), (1, 16, [9], 128, True), (4, 4, [1, 1, 40], 256, False), (8, 8, [60], 128, False)])
def test_a_workspace_of_just_its_bytes_is_enough_for_split_rows(H, Hq, news, D, e4m3):
    c = Cache([2000 + 700 * i for i in range(len(news))], H, D, 64, e4m3).fill()
    T, nB = sum(news), len(news)
    args, q = c.device(), queries(T, Hq, D)
    st = torch.tensor([0, *torch.tensor(news).cumsum(0).tolist()], dtype=torch.int32)
    bytes_ = F.attention_workspace_bytes(T, nB, Hq, H, D)
    memory = torch.full((bytes_ + (8 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    got = F.fp4_attention_prompt(q.cuda(), *args, st.cuda(), workspace=memory[:bytes_], **c.more)
    want, tol = attention(c, q, st.tolist(), D ** -0.5)
    check(got, want, tol, f"prompt rows {news} heads {Hq}/{H} of {D}")
    assert (memory[bytes_:] == 0xA5).all()


@pytest.mark.parametrize("H,Hq,nB,layout,e4m3", [(12, 12, 169, "heads", False), (24, 24, 85, "tokens", False), (20, 40, 101, "tokens", True),
                                                 (1, 4, 300, "heads", True)])
def test_many_short_sequences_with_room_for_long_ones(H, Hq, nB, layout, e4m3):
    """Cut and joined, as the table could hold long ones; and a workspace of just its bytes is enough then too."""
    D = 64
    c = Cache([97 + (37 * b) % 120 if b % 9 else b % 3 for b in range(nB)], H, D, 16, e4m3, layout, cols_more=300).fill()
    args, q = c.device(), queries(nB, Hq, D)
    bytes_ = F.attention_workspace_bytes(nB, nB, Hq, H, D)
    memory = torch.full((bytes_ + (8 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    got = F.fp4_attention_decode(q.cuda(), *args, workspace=memory[:bytes_], **c.more)
    want, tol = attention(c, q, range(nB + 1), D ** -0.5)
    check(got, want, tol, f"decode {nB} sequences heads {Hq}/{H} {layout}")
    assert (memory[bytes_:] == 0xA5).all()


@pytest.mark.parametrize("D,Hq,H,e4m3,layout", [(64, 64, 8, False, "heads"), (128, 32, 8, True, "heads"), (128, 64, 8, True, "tokens"), (256, 4, 4, False, "heads")])
def test_short_sequences_are_not_cut(D, Hq, H, e4m3, layout):
    """Sequences that a workgroup takes whole: by their table, and by a window that fills the GPU with them."""
    run(Cache([1, 0, 15, 33, 64, 97, 120, 128], H, D, 16, e4m3, layout, cols_more=0).fill(), Hq)
    c = Cache([0, 1, 30, 260, 900, 1500, *(700 + 31 * i for i in range(31))], H, D, 16, e4m3, layout).fill()
    run(c, Hq, window=200, sinks=5)


def test_long_decode_is_split():
    for e4m3 in (False, True):
        c = Cache([20000, 3, 4097], 1, 64, 64, e4m3).fill()
        run(c, 2)
        run(c, 2, window=9001, sinks=70)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,Hq,H,window,sinks", [(64, 64, 4, 0, 0), (64, 66, 2, 150, 20), (128, 64, 64, 0, 0), (128, 64, 8, 333, 0)])
def test_rows_that_fill_the_gpu(D, Hq, H, window, sinks, e4m3):
    """More than 256 rows for every CU: the tiles of 256 rows."""
    c = Cache([900, 70, 520, 1], H, D, 32, e4m3, "tokens").fill()
    run(c, Hq, [600, 70, 400, 1], window=window, sinks=sinks, pad=2)


def test_few_rows_over_a_long_cache():
    c = Cache([9000, 5000], 2, 128, 64, True).fill()
    run(c, 8, [3, 17])
    run(c, 8, [3, 17], window=4000, sinks=9)


@pytest.mark.parametrize("e4m3", [False, True])
def test_one_row_prompts_and_decode_agree(e4m3):
    """The same formula through both calls: each within its tolerance of the other's."""
    c = Cache([300, 17, 1000], 2, 128, 16, e4m3).fill()
    q = queries(3, 8, 128)
    args = c.device()
    a = F.fp4_attention_decode(q.cuda(), *args, **c.more)
    b = F.fp4_attention_prompt(q.cuda(), *args, torch.arange(4, dtype=torch.int32).cuda(), **c.more)
    _, tol = attention(c, q, range(4), 128 ** -0.5)
    assert ((a.double() - b.double()).abs().cpu() <= 2 * tol).all()


def test_append_then_attend():
    """A conversation as it is used: a prompt, then token after token, over one cache; each step against float64 on what the cache
    holds then."""
    for e4m3 in (False, True):
        H, Hq, D, S = 2, 8, 64, 16
        prompt, steps = [37, 5, 64], 4
        c = Cache([n + steps for n in prompt], H, D, S, e4m3, "both")
        args = c.device()
        freqs = (1e4 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
        done = [0] * 3
        for step in range(steps + 1):
            news = prompt if step == 0 else [1] * 3
            done = [a + b for a, b in zip(done, news)]
            T = sum(news)
            st = torch.tensor([0, *torch.tensor(news).cumsum(0).tolist()], dtype=torch.int32)
            x = torch.randn(T, Hq + 2 * H, D, generator=torch.Generator().manual_seed(step)).bfloat16().cuda()
            args[3].copy_(torch.tensor(done))
            q = F.fp4_kv_append(x[:, Hq:Hq + H], x[:, Hq + H:], *args, st.cuda() if step == 0 else None, q=x[:, :Hq], freqs=freqs,
                                **c.more)
            got = F.fp4_attention_prompt(q, *args, st.cuda(), **c.more) if step == 0 else F.fp4_attention_decode(q, *args, **c.more)
            # what the cache says it holds
            c.lengths = torch.tensor(done, dtype=torch.int32)
            kp, vp = (t.float().cpu().double() for t in args[:2])
            if e4m3:
                kp, vp = kp * c.more["k_scales"].cpu().double()[..., None], vp * c.more["v_scales"].cpu().double()[..., None]
            c.keys, c.values = [], []
            for b, n in enumerate(done):
                i = torch.arange(n)
                p = c.table[b].long()[i // S]
                c.keys.append(kp[p, :, i % S])
                c.values.append(vp[p, :, i % S])
            want, tol = attention(c, q.cpu(), st.tolist(), D ** -0.5)
            check(got, want, tol, f"step {step}")


def test_wrong_operands_are_refused():
    c, o = Cache([20, 30], 2, 64, 16).fill(), Cache([20, 30], 2, 64, 16, True).fill()
    k, v, table, lengths = c.device()
    ok, ov, _, _ = o.device()
    q = queries(2, 4, 64).cuda()
    st = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    out = torch.full((2, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(F.attention_workspace_bytes(2, 2, 4, 2, 64), dtype=torch.uint8, device="cuda")

    def call(fn, q=q, k=k, v=v, t=table, n=lengths, out=out, **more):
        return fn(q, k, v, t, n, out=out, **more)
    for fn, extra in ((F.fp4_attention_decode, {}), (F.fp4_attention_prompt, dict(starts=st))):
        bad = [dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(q=q[0]), dict(q=q.cpu()), dict(k=ok, v=ov), dict(v=v[:1]),
               dict(k=k.float(), v=v.float()), dict(t=table.long()), dict(n=lengths[:1]), dict(out=out[:1]), dict(out=out.float()),
               dict(workspace=ws[:-1]), dict(workspace=None), dict(workspace=ws.view(torch.int8)), dict(out=out[:, ::2])]
        bad += [dict(starts=None), dict(starts=st[:2]), dict(starts=st.long())] if extra else [dict(q=queries(3, 4, 64).cuda())]
        for i, b in enumerate(bad):
            with pytest.raises(ValueError):
                call(fn, **{**extra, **b})
                pytest.fail(f"{fn.__name__} {i} was not refused")
        for b in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(window=-1), dict(sinks=-3)):
            with pytest.raises(F.Fp4Error):
                call(fn, **{**extra, **b})
    torch.cuda.synchronize()
    assert (out == 7).all()
