"""fp4_kv_append against float64 on the CPU: the rotation, both kinds of cache, every order of memory, and nothing written anywhere
else.

Tolerances: the rotation's float32 error (paged_plain.rotate) and half a step of what holds the result: bf16 2^-8, E4M3 2^-4 of a
value or, below 2^-6 of a code, 2^-10 codes, each by its scale. A scale is three float32 roundings off. What is not rotated is
compared bit for bit.
"""
import pytest
import torch

import microscaling_fp4_quantized_amd as F
import paged_plain
from microscaling_fp4_quantized_amd import binding as B
from paged_plain import Cache
from parity import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


def bits(t):
    return t.contiguous().view(torch.uint8)


def inputs(T, Hq, H, D, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T + pad, Hq + 2 * H, D, generator=g) * 3).bfloat16()
    return x, x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]


def check_close(got, want, tol):
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol.clamp_min(1e-300)).max()))


def run(c, news, Hq, rotated, interleaved=False, positions=None, axes=None, freqs=None, pad=0, seed=3, starts=True, with_q=True):
    """The call on a fresh copy of cache c, and all that it has to have done."""
    H, D, T = c.H, c.D, sum(news)
    x, q, k, v = inputs(T, Hq, H, D, seed, pad)
    st = torch.tensor([0, *torch.tensor(news).cumsum(0).tolist()], dtype=torch.int32)
    if freqs is None and rotated:
        freqs = (1e4 ** (-torch.arange(rotated // 2, dtype=torch.float64) * 2 / rotated)).float()
    args = c.device()
    xd = x.cuda()
    qd, kd, vd = xd[:, :Hq], xd[:, Hq:Hq + H], xd[:, Hq + H:]
    out = torch.full((T + pad, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda") if with_q and rotated else None
    got = F.fp4_kv_append(kd, vd, *args, st.cuda() if starts else None, q=qd if out is not None else None,
                          freqs=freqs.cuda() if rotated else None, positions=None if positions is None else positions.cuda(),
                          axes=None if axes is None else axes.cuda(), interleaved=interleaved, out=out, **c.more)
    torch.cuda.synchronize()
    assert got is out
    assert torch.equal(bits(xd.cpu()), bits(x))
    where = [(b, n - m + r) for b, (n, m) in enumerate(zip(c.lengths.tolist(), news)) for r in range(m)]
    if rotated:
        if positions is None:
            pos = torch.tensor([i for _, i in where], dtype=torch.float64)[:, None].expand(T, rotated // 2)
        else:
            p = positions.view(-1, T + pad)[:, :T].double()
            a = torch.zeros(rotated // 2, dtype=torch.long) if axes is None else axes.long()
            pos = torch.where(((a >= 0) & (a < len(p)))[None], p[a.clamp(0, len(p) - 1)].t(), 0.0)
        angle = pos * freqs.double()
        (kr, kt), (qr, qt) = (paged_plain.rotate(t[:T].double(), angle, interleaved) for t in (k, q))
    else:
        (kr, kt), qr = (k[:T].double(), torch.zeros(T, H, D, dtype=torch.float64)), None
    if out is not None:
        check_close(out[:T].cpu().double(), qr, qt + 2.0 ** -8 * (qr.abs() + qt))
        assert (out[T:] == 7).all()
    # the cache: a copy with the written places taken from what came back
    store, scales = c.on.cpu(), c.scales_on.cpu() if c.e4m3 else None
    view = lambda like, s: s.as_strided(like.shape, like.stride(), like.storage_offset())  # noqa: E731
    held = [(t, *c.place(b, i)) for t, (b, i) in enumerate(where)
            if 0 <= i < c.table.shape[1] * c.S and 0 <= c.place(b, i)[0] < c.P]
    if held:
        t, p, o = torch.tensor(held).unbind(1)
        for like, sc_like, want, tol, x32 in ((c.k, c.ks, kr, kt, None), (c.v, c.vs, v[:T].double(), None, v[:T].float())):
            g = view(like, store)[p, :, o]
            if not c.e4m3:
                if tol is None or not rotated:
                    assert torch.equal(bits(g), bits(want[t].bfloat16()))
                else:
                    check_close(g.double(), want[t], tol[t] + 2.0 ** -8 * (want[t].abs() + tol[t]))
            else:
                s = view(sc_like, scales)[p, :, o]
                if tol is None or not rotated:
                    wc, ws = paged_plain.quantize(want[t].float())
                    assert torch.equal(bits(g), bits(wc)) and torch.equal(bits(s), bits(ws))
                else:
                    top = want[t].abs().amax(-1)
                    check_close(s.double() * 448, top, tol[t].amax(-1) + 2.0 ** -21 * top)
                    val = g.view(paged_plain.E4M3).float().double() * s.double()[..., None]
                    check_close(val, want[t], 2 * tol[t] + (2.0 ** -4 + 2.0 ** -20) * want[t].abs() + 2.0 ** -10 * s.double()[..., None])
            view(like, store)[p, :, o] = like[p, :, o]
            if c.e4m3:
                view(sc_like, scales)[p, :, o] = sc_like[p, :, o]
    assert torch.equal(bits(store), bits(c.store))
    if c.e4m3:
        assert torch.equal(bits(scales), bits(c.scale_store))


LAYOUTS = ["heads", "tokens", "both", "gaps"]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_one_token_each(D, e4m3, layout):
    lengths = [1, 16, 17, 33, 100, 257]
    say(f"append one token, D {D} e4m3 {e4m3} {layout}")
    run(Cache(lengths, 3, D, 16, e4m3, layout), [1] * 6, 6, D, starts=False)
    run(Cache(lengths, 3, D, 32, e4m3, layout), [1] * 6, 6, D // 2, interleaved=True, pad=2)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotated", [0, 16, 48, None])
def test_prompts(D, e4m3, interleaved, rotated):
    news = [1, 130, 0, 61, 7]
    lengths = [1, 130, 40, 200, 7]
    rotated = D if rotated is None else rotated
    say(f"append prompts, D {D} e4m3 {e4m3} interleaved {interleaved} rotated {rotated}")
    run(Cache(lengths, 2, D, 64, e4m3, "tokens", seed=1), news, 4, rotated, interleaved, pad=3)


@pytest.mark.parametrize("Hq,H", [(1, 1), (5, 1), (40, 40), (13, 13)])
def test_heads(Hq, H):
    say(f"append heads {Hq} {H}")
    for e4m3 in (False, True):
        run(Cache([50, 3], H, 64, 16, e4m3), [20, 3], Hq, 64)
        run(Cache([50, 3], H, 64, 16, e4m3), [20, 3], Hq, 64, with_q=False)


@pytest.mark.parametrize("axes", [None, [0, 1, 2], [2, -1, 7]])
def test_axes(axes):
    """Positions of their own, up to the largest there are; a frequency of no axis is not rotated."""
    T, half = 37, 32
    pos = torch.randint(0, 2 ** 31 - 1, (3, T), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    a = None if axes is None else torch.tensor(axes, dtype=torch.int32).repeat(half)[:half].contiguous()
    say(f"append axes {axes}")
    run(Cache([40, 20], 2, 64, 16), [30, 7], 4, 64, positions=pos, axes=a)
    run(Cache([40, 20], 2, 64, 16), [30, 7], 4, 64, positions=-pos[0].contiguous())


def test_far_positions():
    """A million tokens on, at a frequency of 1: float32 angles would be off by 0.03."""
    c = Cache([64], 1, 128, 64, cols_more=0)
    c.lengths[0] = 2 ** 20 + 11
    c.table = torch.full((1, 2 ** 14 + 1), 0, dtype=torch.int32)
    say("append far positions")
    run(c, [5], 2, 128, freqs=torch.linspace(1.0, 3.0, 64))


def test_rows_of_nobody_and_pages_that_are_none():
    c = Cache([100, 100, 100], 2, 64, 16)
    c.table[0, 5] = -1          # tokens 80..95 of sequence 0
    c.table[1, 6] = c.P         # 96..99 of sequence 1
    c.lengths[2] = 3            # of 7 new tokens four stand before the sequence
    say("append, bad pages")
    run(c, [30, 10, 7], 2, 64, pad=5)
    c = Cache([20, 30], 2, 64, 16, cols_more=0)
    c.lengths[0] = 10 ** 9      # past what the table has room for
    run(c, [4, 4], 2, 64)
    c.lengths[0] = -5
    run(c, [4, 4], 2, 64)


def test_many_sequences():
    """More than a wave's lanes of them, some without rows."""
    news = [i % 4 for i in range(200)]
    lengths = [n + i % 9 for i, n in enumerate(news)]
    say("append 200 sequences")
    run(Cache(lengths, 1, 64, 16), news, 1, 64, pad=9)
    run(Cache([i % 50 + 1 for i in range(130)], 1, 64, 16, True), [1] * 130, 1, 64, starts=False)


def test_zeros_and_non_finite():
    """E4M3: a token's zeros get a small scale, a NaN makes its head NaN, an infinity a scale of infinity; no other head changes."""
    c = Cache([8], 3, 64, 16, True)
    args = c.device()
    x = torch.randn(8, 3, 64, generator=torch.Generator().manual_seed(0)).bfloat16()
    x[1, 0] = 0
    x[2, 1, 5] = float("nan")
    x[3, 2, 9] = float("inf")
    F.fp4_kv_append(x.cuda(), x.cuda(), *args, torch.tensor([0, 8], dtype=torch.int32).cuda(), **c.more)
    page = int(c.table[0, 0])
    for pages, scales in ((args[0], c.more["k_scales"]), (args[1], c.more["v_scales"])):
        got = pages[page].float().cpu() * scales[page].cpu()[..., None]  # [heads, places, dims]
        wc, ws = paged_plain.quantize(x.float())
        want = (wc.float() * ws[..., None]).transpose(0, 1)
        fine = torch.ones(3, 8, dtype=torch.bool)
        fine[1, 2] = fine[2, 3] = False
        assert torch.equal(got[:, :8][fine], want[fine])
        assert got[1, 2].isnan().all() and got[2, 3, 9].isnan() and scales[page, 2, 3].isinf()
        assert (scales[page, 0, 1] > 0).item() and (got[0, 1] == 0).all()


def test_queries_in_place():
    """q rotated in the projection's own output: the same bits as into a buffer of its own."""
    x, q, k, v = inputs(21, 4, 2, 128, 1)
    c = Cache([21], 2, 128, 16)
    freqs = (1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    st = torch.tensor([0, 21], dtype=torch.int32).cuda()
    args = c.device()
    xd = x.cuda()
    want = F.fp4_kv_append(xd[:, 4:6], xd[:, 6:], *args, st, q=xd[:, :4], freqs=freqs)
    got = F.fp4_kv_append(xd[:, 4:6], xd[:, 6:], *args, st, q=xd[:, :4], freqs=freqs, out=xd[:, :4])
    assert got.data_ptr() == xd.data_ptr() and torch.equal(bits(got), bits(want))
    assert torch.equal(bits(xd[:, 4:].cpu()), bits(x[:, 4:]))


def test_wrong_operands_are_refused():
    c, o = Cache([20, 30], 2, 64, 16), Cache([20, 30], 2, 64, 16, True)
    k_pages, v_pages, table, lengths = c.device()
    ok, ov, _, _ = o.device()
    x, q, k, v = (t.cuda() for t in inputs(7, 4, 2, 64, 1))
    st = torch.tensor([0, 3, 7], dtype=torch.int32).cuda()
    fr = torch.ones(32).cuda()
    pos = torch.zeros(3, 7, dtype=torch.int32).cuda()
    ax = torch.zeros(32, dtype=torch.int32).cuda()
    before = bits(c.on).clone()

    def call(k=k, v=v, kp=k_pages, vp=v_pages, t=table, n=lengths, s=st, **more):
        return F.fp4_kv_append(k, v, kp, vp, t, n, s, **more)
    bad = [
        dict(k=k.float()), dict(k=k[:, :1]), dict(v=v[:6]), dict(v=v[..., :32]), dict(k=k.cpu()), dict(k=k.transpose(1, 2)),
        dict(kp=ok), dict(kp=ok, vp=ov), dict(vp=v_pages[:1]), dict(vp=v_pages.clone().transpose(1, 2).contiguous().transpose(1, 2)),
        dict(kp=k_pages[0]), dict(k_scales=o.more["k_scales"], v_scales=o.more["v_scales"]),
        dict(kp=ok, vp=ov, k_scales=o.more["k_scales"], v_scales=o.more["v_scales"][:1]),
        dict(kp=ok, vp=ov, k_scales=o.more["k_scales"], v_scales=o.more["v_scales"].double()),
        dict(t=table.long()), dict(t=table[0]), dict(t=table.t()), dict(n=lengths[:1]), dict(n=lengths.long()), dict(n=lengths.cpu()),
        dict(s=st[:2]), dict(s=st.long()), dict(s=None), dict(q=q), dict(positions=pos), dict(axes=ax), dict(freqs=fr, axes=ax),
        dict(freqs=fr.double()), dict(freqs=fr[None]), dict(freqs=fr, positions=pos[:, :6].contiguous()),
        dict(freqs=fr, positions=pos.long()), dict(freqs=fr, positions=pos, axes=ax[:31]), dict(freqs=fr, q=q[:6]),
        dict(freqs=fr, q=q[..., :32]), dict(freqs=fr, q=q, out=q[:, :3]), dict(freqs=fr, out=q), dict(freqs=fr, q=q, out=q.float()),
    ]
    for i, b in enumerate(bad):
        with pytest.raises(ValueError):
            call(**b)
            pytest.fail(f"call {i} was not refused")
    for b in (dict(freqs=fr[:7]), dict(freqs=torch.ones(40).cuda()), dict(k=torch.zeros(7, 2, 68, device="cuda").bfloat16()[..., 4:]),
              dict(freqs=fr, q=q, out=torch.zeros(7, 4, 68, device="cuda").bfloat16()[..., :64])):
        with pytest.raises(F.Fp4Error):
            call(**b)
    torch.cuda.synchronize()
    assert torch.equal(bits(c.on), before)
