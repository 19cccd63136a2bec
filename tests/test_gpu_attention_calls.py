"""How the paged cache's calls are made: compiled and Python checks give the same bits, side streams and replayed graphs those of one call
after another, large operands those of small ones.

(The results themselves are checked against float64 by test_gpu_kv_append.py and test_gpu_attention.py.)
"""
import pytest
import torch

import microscaling_fp4_quantized_amd as F
from microscaling_fp4_quantized_amd import binding as B
from parity import say

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def bits(t):
    return t.contiguous().view(torch.uint8)


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


class Talk:
    """B conversations over a cache of their own: a prompt, then tokens one by one; given outputs and workspaces throughout."""

    def __init__(self, seed, e4m3, Bn=3, Hq=8, H=2, D=64, S=16, most=400):
        self.Hq, self.H, self.D, self.e4m3, self.Bn = Hq, H, D, e4m3, Bn
        cols = -(-most // S)
        g = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(Bn * cols, generator=g).to(torch.int32).view(Bn, cols).to(DEV)
        kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        self.k, self.v = (torch.zeros(Bn * cols, H, S, D, device=DEV).to(kind) for _ in range(2))
        self.more = {n: torch.zeros(Bn * cols, H, S, device=DEV) for n in ("k_scales", "v_scales")} if e4m3 else {}
        self.lengths = torch.zeros(Bn, dtype=torch.int32, device=DEV)
        self.freqs = (1e4 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)).float().to(DEV)
        self.news = [5, 130, 41]
        T = sum(self.news)
        self.starts = torch.tensor([0, 5, 135, 176], dtype=torch.int32, device=DEV)
        self.prompt = normal(seed + 1, T, Hq + 2 * H, D)
        self.token = normal(seed + 2, Bn, Hq + 2 * H, D)
        self.qp, self.op = (torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.qt, self.ot = (torch.empty(Bn, Hq, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.ws = torch.empty(max(F.attention_workspace_bytes(t, Bn, Hq, H, D) for t in (T, Bn)), dtype=torch.uint8, device=DEV)

    def cache(self):
        return self.k, self.v, self.table, self.lengths

    def first(self):
        x, Hq, H = self.prompt, self.Hq, self.H
        F.fp4_kv_append(x[:, Hq:Hq + H], x[:, Hq + H:], *self.cache(), self.starts, q=x[:, :Hq], freqs=self.freqs, out=self.qp, **self.more)
        F.fp4_attention_prompt(self.qp, *self.cache(), self.starts, window=100, sinks=3, out=self.op, workspace=self.ws, **self.more)

    def step(self):
        x, Hq, H = self.token, self.Hq, self.H
        F.fp4_kv_append(x[:, Hq:Hq + H], x[:, Hq + H:], *self.cache(), q=x[:, :Hq], freqs=self.freqs, out=self.qt, **self.more)
        F.fp4_attention_decode(self.qt, *self.cache(), out=self.ot, workspace=self.ws, **self.more)

    def run(self):
        self.lengths.copy_(torch.tensor(self.news, dtype=torch.int32))
        self.first()
        for _ in range(2):
            self.lengths += 1
            self.step()

    def outputs(self):
        return [self.k, self.v, *self.more.values(), self.qp, self.op, self.qt, self.ot]

    def copies(self):
        return [bits(t).clone() for t in self.outputs()]

    def clear(self):
        for t in self.outputs():
            t.view(torch.uint8).fill_(0x55)


def same(talk, want):
    return [i for i, (t, w) in enumerate(zip(talk.outputs(), want)) if not torch.equal(bits(t), w)]


def done(talk):
    torch.cuda.synchronize()
    return talk.copies()


def test_the_compiled_checks_are_built_and_used():
    fast = B._fast(torch.empty(1, device=DEV))
    assert fast and fast.append and fast.decode and fast.prompt


@pytest.mark.parametrize("e4m3", [False, True])
def test_compiled_and_python_checks_give_the_same_bits(e4m3, monkeypatch):
    say(f"attention calls e4m3 {e4m3}")
    talk = Talk(1, e4m3)
    talk.clear()
    talk.run()
    want = done(talk)
    monkeypatch.setattr(B, "_FAST", False)
    talk.clear()
    talk.run()
    assert not same(talk, done(talk)) and not same(talk, want)
    # and with outputs and workspaces of the calls' own
    q = F.fp4_kv_append(talk.token[:, 8:10], talk.token[:, 10:], *talk.cache(), q=talk.token[:, :8], freqs=talk.freqs, **talk.more)
    assert torch.equal(bits(q), want[-2])
    assert torch.equal(bits(F.fp4_attention_decode(q, *talk.cache(), **talk.more)), want[-1])


def test_a_module_without_these_calls_serves_the_others(monkeypatch):
    import types
    from microscaling_fp4_quantized_amd import _torch_calls as module
    old = types.SimpleNamespace(**{n: getattr(module, n) for n in ("quantize", "norm", "linear", "route", "experts")})
    fast = B._Fast(old, B.load_library())
    assert fast.append is None and fast.decode is None and fast.prompt is None
    talk = Talk(4, False)
    talk.clear()  # the places that no call writes, too
    talk.run()
    want = done(talk)
    monkeypatch.setattr(B, "_FAST", fast)
    talk.clear()
    talk.run()
    torch.cuda.synchronize()
    assert not same(talk, want)


@pytest.mark.parametrize("e4m3", [False, True])
def test_side_streams_match_serial(e4m3):
    say(f"attention on two streams, e4m3 {e4m3}")
    talks = [Talk(10 * i, e4m3) for i in range(4)]
    want = []
    for t in talks:
        t.clear()
        t.run()
        want.append(done(t))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for t in talks:
            t.clear()
        torch.cuda.synchronize()
        for i, t in enumerate(talks):
            with torch.cuda.stream(streams[i % 2]):
                t.run()
        torch.cuda.synchronize()
        assert [same(t, w) for t, w in zip(talks, want)] == [[]] * 4


@pytest.mark.parametrize("e4m3", [False, True])
def test_graph_replays_follow_the_lengths(e4m3):
    """A captured step reads the lengths and the table when it is replayed: each replay is the eager step on what they hold then. Two graphs
    share the workspace, one after the other."""
    say(f"attention in graphs, e4m3 {e4m3}")
    talk, eager = Talk(1, e4m3), Talk(1, e4m3)
    for t in (talk, eager):
        t.clear()
        t.run()
    eager.first()
    eager.step()  # as talk does before its capture
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        talk.first()
        talk.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    first, step = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        talk.first()
    with torch.cuda.graph(step):
        talk.step()
    for rep in range(4):
        for t in (talk, eager):
            t.lengths.copy_(torch.tensor([5 + rep, 200 - 9 * rep, 41], dtype=torch.int32))
            t.table.copy_(t.table.flip(0))
            t.token.mul_(-1)
        first.replay()
        eager.first()
        torch.cuda.synchronize()
        for t in (talk, eager):
            t.lengths += 100
        step.replay()
        eager.step()
        torch.cuda.synchronize()
        assert not same(talk, eager.copies()), rep


def near(a, b):
    a, b = a.double(), b.double()
    return bool((a - b).norm() <= 2.0 ** -8 * b.norm()) and bool(b.norm() > 0)


@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_past_2_32_bytes(e4m3):
    """The last pages of a cache of more than 4 GiB (8-bit: codes), and scales past 2^31: written and read as those of a small one."""
    H, S, D = 8, 64, 128
    P = (1 << 32) // (H * S * D * (1 if e4m3 else 2)) + 77
    say(f"cache of {P} pages")
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    lengths = torch.tensor([200, 64], dtype=torch.int32, device=DEV)
    x = normal(3, 264, 32 + 16, D)
    starts = torch.tensor([0, 200, 264], dtype=torch.int32, device=DEV)
    got = []
    for pages, table in ((P, [[P - 1, P - 2, 0, P - 4], [P - 5, 0, 0, 0]]), (9, [[8, 7, 0, 5], [4, 0, 0, 0]])):
        k, v = (torch.empty(pages, H, S, D, dtype=kind, device=DEV) for _ in range(2))
        more = {n: torch.empty(pages, H, S, device=DEV) for n in ("k_scales", "v_scales")} if e4m3 else {}
        t = torch.tensor(table, dtype=torch.int32, device=DEV)
        F.fp4_kv_append(x[:, 32:40], x[:, 40:], k, v, t, lengths, starts, **more)
        q = x[:, :32]
        got.append((F.fp4_attention_prompt(q, k, v, t, lengths, starts, **more), F.fp4_attention_decode(q[:2], k, v, t, lengths, **more)))
        torch.cuda.synchronize()
        del k, v, more
        torch.cuda.empty_cache()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(*got)) and all(a.isfinite().all() and a.any() for a in got[0])


def test_rows_past_2_31_elements():
    """Queries and outputs of more than 2^31 elements, streamed past the caches: the last rows as in a call of their own."""
    H, S, D, Hq, tail = 1, 64, 128, 128, 300
    T = (1 << 31) // (Hq * D) + 5000
    say(f"{T} rows of {Hq} heads")
    cols = -(-T // S)
    table = torch.full((2, cols), -1, dtype=torch.int32, device=DEV)
    table[0] = torch.arange(cols)
    table[1, :8] = torch.arange(cols, cols + 8)
    k, v = (torch.empty(cols + 8, H, S, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    lengths = torch.tensor([T - tail, tail], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, T - tail, T], dtype=torch.int32, device=DEV)
    q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(1))
    kv = torch.empty(T, 2, D, dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(2))
    freqs = torch.linspace(1, 1e-4, 64, device=DEV)
    out = F.fp4_kv_append(kv[:, :1], kv[:, 1:], k, v, table, lengths, starts, q=q, freqs=freqs)
    at = F.fp4_attention_prompt(out, k, v, table, lengths, starts, window=200)
    del k, v
    k, v = (torch.empty(8, H, S, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    one = (torch.arange(8, dtype=torch.int32, device=DEV)[None].contiguous(), lengths[1:].clone())
    st = torch.tensor([0, tail], dtype=torch.int32, device=DEV)
    want = F.fp4_kv_append(kv[-tail:, :1], kv[-tail:, 1:], k, v, *one, st, q=q[-tail:], freqs=freqs)
    assert torch.equal(bits(out[-tail:]), bits(want))
    assert near(at[-tail:], F.fp4_attention_prompt(want, k, v, *one, st, window=200))
