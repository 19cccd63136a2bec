"""Attention over a paged key-value cache next to the projections that feed it: cases, plain forms and exact values.

A cache holds pages of `page` tokens, [P, Hkv, page, D], in bf16 or in 8 bits (E4M3 with one float32 scale for a token's D
values of a head). Row b of `table` names the pages of sequence b in order, lengths[b] says how many tokens it holds, the new ones
among them; new token t of sequence b, starts[b] <= t < starts[b + 1], stands at i = lengths[b] - (starts[b + 1] - t).

    append  k, v -> the cache at i; q and k rotated on the way: pairs (a, b) -> (a cos w - b sin w, a sin w + b cos w) with
            w = position * frequency, the position i itself or one of several axes (time, height, width) for each frequency
    decode  one new token of each sequence: o_h = sum_j softmax_j(scale q_h k_j) v_j over the visible j
    prompt  the same for every new token, which stand in rows starts[b] .. starts[b + 1]

visible: j <= i and (no window, or i - j < window, or j < sinks).

`run` computes a case in plain torch operations in float32, or with `own` through the framework's operators.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # a token of zeros still has a finite scale
SCORES = 1 << 28          # elements of a score matrix that the plain forms hold at once


def listed():
    def case(name, op, B, cached, new, Hq, Hkv, D, page, e4m3, layout="heads", mix=1, **more):
        return {"name": name, "op": op, "B": B, "cached_least": cached[0], "cached_most": cached[1], "new_least": new[0],
                "new_most": new[1], "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "e4m3": e4m3, "layout": layout, "mix": mix, **more}

    return [
        # one token of one conversation: a latency
        case("append_token", "append", 1, (1000, 1000), (1, 1), 32, 8, 128, 64, False, R=128, interleaved=False, axes=1, pad=0),
        # an odd decode batch over an 8-bit cache, far positions, half of a head's values rotated
        case("append_batch", "append", 61, (100, 8000), (1, 1), 64, 8, 64, 16, True, R=32, interleaved=True, axes=1, pad=3),
        # a few images and their texts: positions of three axes
        case("append_axes", "append", 3, (0, 40), (300, 1600), 16, 2, 128, 16, False, "tokens", R=128, interleaved=False, axes=3,
             pad=0),
        # many prompts at once into an 8-bit cache: bound by memory
        case("append_prompts", "append", 9, (0, 900), (700, 6000), 32, 8, 128, 64, True, R=128, interleaved=False, axes=1, pad=64),
        # one token of one conversation
        case("decode_token", "decode", 1, (1000, 1000), (1, 1), 32, 8, 128, 64, False, window=0, sinks=0),
        # one token of a long document: the length has to be split
        case("decode_long", "decode", 1, (131000, 131000), (1, 1), 32, 8, 128, 64, False, window=0, sinks=0),
        # a ragged batch over an 8-bit cache
        case("decode_batch", "decode", 64, (60, 8100), (1, 1), 64, 8, 128, 32, True, "tokens", window=0, sinks=0),
        # a layer that sees a window and the first tokens, long conversations
        case("decode_window", "decode", 37, (2000, 32000), (1, 1), 64, 8, 64, 16, False, window=1024, sinks=4),
        # a few short questions
        case("prompt_short", "prompt", 7, (0, 0), (1, 150), 32, 8, 128, 64, False, window=0, sinks=0, pad=5),
        # one long document
        case("prompt_long", "prompt", 1, (0, 0), (8192, 8192), 32, 8, 128, 64, False, window=0, sinks=0, pad=0),
        # the same through a layer with a window
        case("prompt_window", "prompt", 3, (0, 0), (2000, 9000), 64, 8, 64, 16, False, "tokens", window=1024, sinks=4, pad=0),
        # the next pieces of two long documents over an 8-bit cache
        case("prompt_piece", "prompt", 2, (9000, 16001), (512, 512), 32, 8, 128, 32, True, window=0, sinks=0, pad=0),
    ]


def _log(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    while True:
        op = rng.choice(["append", "decode", "decode", "prompt", "prompt"])
        Hkv = rng.choice([1, 2, 4, 8, 8, 16])
        case = {"op": op, "Hkv": Hkv, "Hq": Hkv * rng.choice([1, 2, 3, 4, 8, 16]), "D": rng.choice([64, 128, 128, 256]),
                "page": rng.choice([16, 32, 64, 128, 256]), "e4m3": rng.random() < 0.5, "layout": rng.choice(["heads", "tokens"]),
                "mix": rng.randint(1, 1 << 20)}
        if case["Hq"] > 64:
            continue
        if op == "decode":
            case.update(B=_log(rng, 1, 256), cached_most=_log(rng, 1, 131072), new_least=1, new_most=1)
        else:
            case.update(B=_log(rng, 1, 16), cached_most=rng.choice([0, _log(rng, 1, 16384)]), new_most=_log(rng, 1, 8192))
            case.update(new_least=_log(rng, 1, case["new_most"]), pad=rng.choice([0, 0, 1, 17]))
        case["cached_least"] = min(case["cached_most"], _log(rng, 1, max(1, case["cached_most"])))
        if op == "append":
            R = rng.choice([case["D"], case["D"], case["D"] // 2, 16])
            case.update(R=R, interleaved=rng.random() < 0.5, axes=rng.choice([1, 1, 3]))
        else:
            case["window"] = rng.choice([0, 0, _log(rng, 1, 8192)])
            case["sinks"] = rng.choice([0, 1, 4, 100]) if case["window"] else 0
        w, like = work(case), [work(c) for c in listed() if c["op"] == op]
        lengths, new = _lengths(case)
        if all(w[n] <= max(k[n] for k in like) for n in w) and sum(lengths) * Hkv * case["D"] <= 1 << 28 and sum(new) <= 32768:
            return case


def _lengths(case):
    """Tokens in the cache and new ones among them, of each sequence: spread over their logarithm, the first ones the most."""
    rng = random.Random(case["mix"])

    def some(lo, hi):
        return [hi] + [int(round(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1))))) - 1 for _ in range(case["B"] - 1)]
    new = [max(1, n) for n in some(case["new_least"], case["new_most"])]
    cached = some(case["cached_least"], case["cached_most"])
    if case["op"] == "decode" and not case["cached_most"]:
        cached = [0] * case["B"]
    return [c + n for c, n in zip(cached, new)], new


# ---- inputs ----------------------------------------------------------------------------------------------------------

def _heads(g, rows, H, D):
    """bf16 rows of H heads: normal values, 2% of the channels 4 times as large and a part that all rows share, as keys have."""
    x = torch.randn(rows, H, D, generator=g, device="cuda")
    loud = torch.rand(H, D, generator=g, device="cuda") < 0.02
    return ((x + 0.5 * torch.randn(H, D, generator=g, device="cuda")) * torch.where(loud, 4.0, 1.0)).bfloat16()


def _to_e4m3(x):
    """Codes and scales of float32 x, one scale for the values of the last dimension."""
    amax = x.abs().amax(dim=-1).clamp_min(AMAX_FLOOR)
    return (x * (E4M3_MAX / amax)[..., None]).to(torch.float8_e4m3fn), amax / E4M3_MAX


def _pages(g, s, P):
    """A cache of P pages with something in every place, [P, Hkv, page, D] whichever lies next to which in memory."""
    H, S, D = s["Hkv"], s["page"], s["D"]
    shape = (P, S, H, D) if s["layout"] == "tokens" else (P, H, S, D)
    pages, scales = [], []
    for _ in range(2):
        pool = torch.randn(1 << 20, generator=g, device="cuda").bfloat16()
        x = torch.empty(shape, dtype=torch.float8_e4m3fn if s["e4m3"] else torch.bfloat16, device="cuda")
        sc = torch.empty(shape[:3], dtype=torch.float32, device="cuda") if s["e4m3"] else None
        step = max(1, (1 << 25) // (H * S * D))
        for p in range(0, P, step):
            n = min(step, P - p)
            rows = n * H * S
            at = torch.randint(0, (1 << 20) // 64 - D // 64, (rows, 1), generator=g, device="cuda") * 64
            v = pool[at + torch.arange(D, device="cuda")].view(n, *shape[1:])
            if s["e4m3"]:
                x[p:p + n], sc[p:p + n] = _to_e4m3(v.float())
            else:
                x[p:p + n] = v
        if s["layout"] == "tokens":
            x, sc = x.transpose(1, 2), sc.transpose(1, 2) if s["e4m3"] else None
        pages.append(x)
        scales.append(sc)
    return pages, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    op, B, Hq, Hkv, D = (case[n] for n in ("op", "B", "Hq", "Hkv", "D"))
    lengths, new = _lengths(case)
    held = [-(-n // case["page"]) for n in lengths]
    cols, P = max(held) + 1, sum(held) + B + 2
    (s["k_pages"], s["v_pages"]), (s["k_scales"], s["v_scales"]) = _pages(g, s, P)
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"], s["lengths"] = table, torch.tensor(lengths, dtype=torch.int32, device="cuda")
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    T = starts[-1] + case.get("pad", 0)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["host_lengths"], s["host_starts"] = lengths, starts  # a scheduler's own copies: the plain forms' loops
    if op == "append":
        qkv = _heads(g, T, Hq + 2 * Hkv, D)  # one projection's output
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        half = case["R"] // 2
        s["freqs"] = (1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        s["positions"] = s["axes_of"] = None
        if case["axes"] > 1:
            s["positions"] = torch.randint(0, 20000, (case["axes"], T), generator=g, device="cuda", dtype=torch.int32)
            s["axes_of"] = (torch.arange(half, device="cuda") * case["axes"] // half).to(torch.int32)
        s["out"] = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    else:
        rows = B if op == "decode" else T
        s["q"] = _heads(g, rows, Hq, D)
        s["out"] = torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device="cuda")
        s["scale"] = D ** -0.5
        if own:
            import microscaling_fp4_quantized_amd as F
            s["workspace"] = torch.empty(F.attention_workspace_bytes(rows, B, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    return s


# ---- plain forms, in float32 -----------------------------------------------------------------------------------------

def _rotate(x, cos, sin, interleaved):
    half = cos.shape[-1]
    x = x.float()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _plain_append(s):
    S, T = s["page"], s["host_starts"][-1]
    t = torch.arange(T, device="cuda")
    b = torch.bucketize(t, s["starts"][1:].long(), right=True)
    i = s["lengths"].long()[b] - (s["starts"].long()[b + 1] - t)
    at = (s["table"].long()[b, i // S], slice(None), i % S)
    if s["positions"] is None:
        angle = i.double()[:, None] * s["freqs"].double()
    else:
        angle = s["positions"].double()[s["axes_of"].long(), :T].t() * s["freqs"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    s["out"][:T] = _rotate(s["q"][:T], cos, sin, s["interleaved"]).bfloat16()
    k, v = _rotate(s["k"][:T], cos, sin, s["interleaved"]), s["v"][:T]
    if s["e4m3"]:
        for x, pages, scales in ((k, s["k_pages"], s["k_scales"]), (v.float(), s["v_pages"], s["v_scales"])):
            codes, sc = _to_e4m3(x)
            pages.view(torch.uint8)[at] = codes.view(torch.uint8)
            scales[at] = sc
        return s["out"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]
    s["k_pages"][at] = k.bfloat16()
    s["v_pages"][at] = v
    return s["out"], s["k_pages"], s["v_pages"]


def _gather(s, b, j):
    """Keys and values of tokens j of sequences b, in float32: [..., Hkv, D] each."""
    page = s["table"].long()[b, j // s["page"]]
    at = (page, slice(None), j % s["page"])
    if not s["e4m3"]:
        return s["k_pages"][at].float(), s["v_pages"][at].float()
    return tuple(p.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * c[at][..., None]
                 for p, c in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])))


def _seen(s, i, j):
    seen = j <= i
    if s["window"]:
        seen = seen & ((i - j < s["window"]) | (j < s["sinks"]))
    return seen


def _plain_decode(s):
    B, Hq, Hkv, D, w, first = (s[n] for n in ("B", "Hq", "Hkv", "D", "window", "sinks"))
    most = max(s["host_lengths"])
    most = min(most, w + first) if w else most
    step = max(1, SCORES // (most * Hkv * D))
    for b0 in range(0, B, step):
        n = min(step, B - b0)
        i = s["lengths"][b0:b0 + n].long()[:, None] - 1
        j = torch.arange(most, device="cuda").expand(n, most)
        if w:  # past the first tokens, the last ones
            j = torch.where(j < first, j, torch.maximum(j, j + i + 1 - w - first))
        seen = _seen(s, i, j)
        k, v = _gather(s, torch.arange(b0, b0 + n, device="cuda")[:, None], torch.minimum(j, i))  # [n, most, Hkv, D]
        q = s["q"][b0:b0 + n].float().view(n, Hkv, Hq // Hkv, D) * s["scale"]
        z = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous())
        z = z.masked_fill(~seen[:, None, None], -math.inf)
        p = torch.exp(z - z.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        s["out"][b0:b0 + n] = torch.matmul(p, v.transpose(1, 2).contiguous()).view(n, Hq, D).bfloat16()
    return s["out"]


def _plain_prompt(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    G = Hq // Hkv
    for b, (n, t0, t1) in enumerate(zip(s["host_lengths"], s["host_starts"], s["host_starts"][1:])):
        k, v = _gather(s, torch.full((n,), b, device="cuda"), torch.arange(n, device="cuda"))
        k, v = k.permute(1, 2, 0).contiguous(), v.transpose(0, 1).contiguous()  # [Hkv, D, n], [Hkv, n, D]
        step = max(1, SCORES // (Hq * n))
        for t in range(t0, t1, step):
            rows = min(step, t1 - t)
            i = torch.arange(t, t + rows, device="cuda")[:, None] + (n - t1)
            seen = _seen(s, i, torch.arange(n, device="cuda"))
            q = (s["q"][t:t + rows].float() * s["scale"]).view(rows, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * rows, D)
            z = torch.matmul(q, k).view(Hkv, G, rows, n).masked_fill_(~seen, -math.inf)
            p = torch.exp(z - z.amax(-1, keepdim=True))
            p = (p / p.sum(-1, keepdim=True)).view(Hkv, G * rows, n)
            o = torch.matmul(p, v).view(Hkv, G, rows, D)
            s["out"][t:t + rows] = o.permute(2, 0, 1, 3).reshape(rows, Hq, D).bfloat16()
    return s["out"]


def run(s):
    op = s["op"]
    if not own:
        return {"append": _plain_append, "decode": _plain_decode, "prompt": _plain_prompt}[op](s)
    import microscaling_fp4_quantized_amd as F

    cache = (s["k_pages"], s["v_pages"], s["table"], s["lengths"])
    if op == "append":
        F.fp4_kv_append(s["k"], s["v"], *cache, s["starts"], q=s["q"], freqs=s["freqs"], positions=s["positions"],
                        axes=s["axes_of"], interleaved=s["interleaved"], k_scales=s["k_scales"], v_scales=s["v_scales"],
                        out=s["out"])
        return (s["out"], *cache[:2], s["k_scales"], s["v_scales"]) if s["e4m3"] else (s["out"], *cache[:2])
    more = dict(scale=s["scale"], window=s["window"], sinks=s["sinks"], k_scales=s["k_scales"], v_scales=s["v_scales"],
                out=s["out"], workspace=s["workspace"])
    if op == "decode":
        return F.fp4_attention_decode(s["q"], *cache, **more)
    return F.fp4_attention_prompt(s["q"], *cache, s["starts"], **more)


def work(case):
    lengths, new = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    entry = D + 4 if case["e4m3"] else 2 * D  # bytes of a token's key, or value, of a head
    if case["op"] == "append":
        T = sum(new)
        return {"bytes": T * (4 * Hq * D + 4 * Hkv * D + 2 * Hkv * entry + 4 * case["axes"]), "flops": T * 3 * case["R"] * (Hq + Hkv)}
    read, pairs = 0, 0
    for n, m in zip(lengths, new):
        first, w, k = n - m, case["window"] or n, case["sinks"]  # the first new token's place
        read += n - max(0, first - w + 1 - k)
        pairs += _ramp(first, n, w) + _ramp(first - w, n - w, k)  # the window's tokens, and those of the first before them
    return {"bytes": read * 2 * Hkv * entry + 4 * sum(new) * Hq * D, "flops": 4 * pairs * Hq * D}


def _ramp(lo, hi, top):
    """Sum over i in [lo, hi) of min(max(i + 1, 0), top)."""
    def to(n):  # over i in [0, n)
        n = max(0, n)
        return n * (n + 1) // 2 if n <= top else top * (top + 1) // 2 + (n - top) * top
    return to(hi) - to(lo)


# ---- exact values, in 64 bits, before the one rounding of each output ------------------------------------------------

def _exact_pages(pages, scales):
    x = pages.double()
    return x if scales is None else x * scales.double()[..., None]


def _exact_append(s):
    T, D, R, S = s["host_starts"][-1], s["D"], s["R"], s["page"]
    where = []
    for n, t0, t1, row in zip(s["host_lengths"], s["host_starts"], s["host_starts"][1:], s["table"].tolist()):
        where += [(row[i // S], i % S, i) for i in range(n - (t1 - t0), n)]
    page, place, index = torch.tensor(where, device="cuda").unbind(1)
    if s["positions"] is None:
        w = torch.outer(index.double(), s["freqs"].double())
    else:
        w = torch.stack([s["positions"][int(a), :T].double() * f for a, f in zip(s["axes_of"].tolist(), s["freqs"].double())], 1)

    def turned(x):
        x = x[:T].double()
        pair = x[:, :, :R].unflatten(2, (R // 2, 2) if s["interleaved"] else (2, R // 2))
        if not s["interleaved"]:
            pair = pair.transpose(2, 3)
        z = torch.polar(torch.ones_like(w), w)[:, None] * torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous())
        y = torch.view_as_real(z)
        y = (y if s["interleaved"] else y.transpose(2, 3)).reshape(T, -1, R)
        return torch.cat([y, x[:, :, R:]], 2)

    out = s["out"].double()
    out[:T] = turned(s["q"])
    caches, factors = [], []
    for x, pages, scales in ((turned(s["k"]), s["k_pages"], s["k_scales"]), (s["v"][:T].double(), s["v_pages"], s["v_scales"])):
        whole = pages.double()
        if scales is not None:
            sc = scales.double()
            sc[page, :, place] = x.abs().amax(2).clamp(min=AMAX_FLOOR) / E4M3_MAX
            x = x / sc[page, :, place][..., None]
            factors.append(sc)
        whole[page, :, place] = x
        caches.append(whole)
    return (out, *caches, *factors)


def _exact_attention(s):
    S, G, w = s["page"], s["Hq"] // s["Hkv"], s["window"] or max(s["host_lengths"])
    out = s["out"].double()
    starts = range(s["B"] + 1) if s["op"] == "decode" else s["host_starts"]
    for b, n in enumerate(s["host_lengths"]):
        t0, t1 = starts[b], starts[b + 1]
        ids = s["table"][b, :-(-n // S)].long()
        raw = [p.view(torch.uint8)[ids].view(p.dtype) if s["e4m3"] else p[ids] for p in (s["k_pages"], s["v_pages"])]
        k, v = (_exact_pages(r, None if c is None else c[ids]).transpose(0, 1).reshape(s["Hkv"], -1, s["D"])[:, :n]
                for r, c in zip(raw, (s["k_scales"], s["v_scales"])))
        place = torch.arange(n - (t1 - t0), n, device="cuda")
        j = torch.arange(n, device="cuda")
        for h in range(s["Hq"]):
            for r in range(0, t1 - t0, 4096):
                at = place[r:r + 4096, None]
                hidden = (j > at) | ((j <= at - w) & (j >= s["sinks"]))
                z = (s["q"][t0 + r:t0 + r + len(at), h].double() @ k[h // G].t()) * s["scale"]
                e = (z - z.masked_fill(hidden, -1e300).amax(1, keepdim=True)).exp_().masked_fill_(hidden, 0.0)
                out[t0 + r:t0 + r + len(at), h] = (e @ v[h // G]) / e.sum(1, keepdim=True)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)
