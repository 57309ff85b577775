"""Measured cases of a decode step's attention: rotary positions (gf_rope), the 8-bit cache of keys and
values as it is written and read back (gf_cache_store, gf_cache_load) and attention over it (gf_attend).

`run` computes them from elementary torch operations where `own` is false, and through the library where
it is true.  The cache: codes [page][head][token of the page][dim], one byte each, and a 32-bit scale for
every `block` tokens of a page and head, [page][head][block].  Formats: i8, value = scale * int8, scales of
12 significant bits; e4m3, value = scale * e4m3, scales that are powers of two.  Token t of a call is
position pos[t] of sequence seq[t]; a sequence's pages are listed in its row of the page table.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16}
MOST = {"i8": 127.0, "e4m3": 448.0}
SMALLEST, LARGEST = 2.0 ** -112, {"i8": 2.0 ** 121, "e4m3": 2.0 ** 119}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # The queries of one user's token: latency only.
        dict(name="rope_token", op="rope", T=1, H=32, D=128, rot=128, layout="halves", type="f32", base=10000.0,
             scaling="plain", factor=1.0, far=4096),
        # An odd batch in half precision, half of each small head rotated, neighbours paired.
        dict(name="rope_odd", op="rope", T=61, H=25, D=80, rot=40, layout="pairs", type="f16", base=10000.0,
             scaling="linear", factor=4.0, far=16384),
        # A long prompt's queries and keys, far positions of a stretched context.
        dict(name="rope_prompt", op="rope", T=8191, H=40, D=128, rot=128, layout="halves", type="f32", base=500000.0,
             scaling="ramp", factor=16.0, far=131072),
        # One user's token: queries and keys rotated, keys and values written into a started block.
        dict(name="store_token", op="store", seqs=1, new=1, Hq=32, H=8, D=128, fmt="i8", block=16, page=16, type="f16",
             rope="halves", before=1000),
        # A batch of users, a scale for every token.
        dict(name="store_batch", op="store", seqs=61, new=61, Hq=32, H=8, D=128, fmt="e4m3", block=1, page=64,
             type="f16", rope="pairs", before=2000),
        # Ragged prompts without a rotation, 32-bit projections; what comes back is what the codes stand for.
        dict(name="store_prompt", op="store", seqs=7, new=8191, Hq=0, H=8, D=128, fmt="i8", block=32, page=64,
             type="f32", rope="none", before=300),
        # One user, a short context: latency only.
        dict(name="attend_token", op="attend", seqs=1, per=1, pad=0, Hq=32, H=8, D=128, fmt="i8", block=16, page=16,
             type="f32", window=0, shortest=1000, longest=1000),
        # One user, a long context: eight rows of work for the whole card.
        dict(name="attend_long", op="attend", seqs=1, per=1, pad=0, Hq=32, H=8, D=128, fmt="i8", block=16, page=64,
             type="f32", window=0, shortest=131071, longest=131071),
        # A batch of users with contexts of all lengths, and rows that no user has.
        dict(name="attend_batch", op="attend", seqs=61, per=1, pad=3, Hq=32, H=8, D=128, fmt="i8", block=32, page=32,
             type="f32", window=0, shortest=100, longest=8000),
        # Small heads, eight queries to a key head, a scale for every token, half precision.
        dict(name="attend_small_heads", op="attend", seqs=33, per=1, pad=0, Hq=64, H=8, D=64, fmt="e4m3", block=1,
             page=64, type="f16", window=0, shortest=1000, longest=16000),
        # Five drafted tokens of each user at once, large heads, only the last 4096 keys.
        dict(name="attend_drafts", op="attend", seqs=16, per=5, pad=0, Hq=16, H=8, D=256, fmt="i8", block=16, page=64,
             type="f32", window=4096, shortest=2000, longest=10000),
        # The widest batch: the cache is what fills the card.
        dict(name="attend_wide", op="attend", seqs=256, per=1, pad=0, Hq=32, H=8, D=128, fmt="i8", block=64, page=64,
             type="f16", window=0, shortest=4000, longest=8000),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "store", "attend", "attend"))
    D = rng.choice((64, 80, 96, 128, 128, 256))
    typ = rng.choice(("f32", "f32", "f16"))
    fmt = rng.choice(("i8", "i8", "e4m3"))
    if op == "rope":
        T, H = _log_int(rng, 1, 8191), rng.randint(1, 48)
        while T * H * D > 8191 * 40 * 128:
            T //= 2
        scaling = rng.choice(("plain", "linear", "ramp", "bands"))
        return dict(op="rope", T=T, H=H, D=D, rot=rng.choice((D, D, D // 2)), layout=rng.choice(("halves", "pairs")),
                    type=typ, base=rng.choice((10000.0, 500000.0)), scaling=scaling,
                    factor=1.0 if scaling == "plain" else rng.choice((4.0, 8.0, 32.0)), far=_log_int(rng, 1000, 200000))
    page = rng.choice((16, 32, 64, 128))
    block = rng.choice([b for b in (1, 4, 16, 32, 64) if b <= page])
    H = rng.choice((1, 2, 4, 8))
    if op == "store":
        seqs = _log_int(rng, 1, 128)
        rope = rng.choice(("none", "halves", "pairs"))
        new = seqs if rng.random() < 0.5 else _log_int(rng, seqs, 8191)
        Hq = 0 if rope == "none" else H * rng.choice((1, 2, 4))
        while new * (Hq + 2 * H) * D > 8191 * 2 * 8 * 128 and new > seqs:
            new = max(seqs, new // 2)
        return dict(op="store", seqs=seqs, new=new, Hq=Hq, H=H, D=D, fmt=fmt, block=block, page=page,
                    type=typ if rope == "none" else "f16", rope=rope, before=_log_int(rng, 1, 2000))
    seqs = _log_int(rng, 1, 256)
    per = rng.choice((1, 1, 1, 2, 4, 8))
    G = rng.choice((1, 2, 4, 5, 8, 16))
    longest = _log_int(rng, 16, 131072)
    while seqs * longest * H * D * (1 + per * G / 8) > 256 * 6000 * 8 * 128:
        longest = longest // 2 + 8
        seqs = max(1, seqs * 2 // 3)
    return dict(op="attend", seqs=seqs, per=per, pad=rng.choice((0, 0, 3)), Hq=H * G, H=H, D=D, fmt=fmt, block=block,
                page=page, type=typ, window=rng.choice((0, 0, 0, 1000)), shortest=max(per, longest // 8),
                longest=max(per, longest))


def _lengths(case):
    """Keys of each sequence after the step (attend), or before it (store); the case's own, whatever the seed."""
    r = np.random.RandomState(case["seqs"] * 131 + case["D"])
    if case["op"] == "store":
        return r.randint(0, case["before"] + 1, case["seqs"])
    lo, hi = math.log(case["shortest"]), math.log(case["longest"])
    return np.exp(r.uniform(lo, hi, case["seqs"])).round().astype(np.int64).clip(case["shortest"], case["longest"])


def _news(case):
    """New tokens of each sequence (store): one at least, a ragged rest."""
    n, extra = case["seqs"], case["new"] - case["seqs"]
    r = np.random.RandomState(case["new"] * 17 + n)
    cuts = np.sort(r.randint(0, extra + 1, n - 1)) if n > 1 else np.zeros(0, dtype=np.int64)
    return 1 + np.diff(np.concatenate(([0], cuts, [extra])))


# ------------------------------------------------------------------ inputs

def _freqs(case, n):
    """The n rotated pairs' angles of one position, in 64 bits, and the factor of cosine and sine."""
    base, factor, scaling, span = case.get("base", 10000.0), case.get("factor", 1.0), case.get("scaling", "plain"), 8192.0
    i = np.arange(n)
    f = base ** (-i / n)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ramp":  # from the pair that turns 32 times over the old span to the one that turns once
        def where(turns):
            return n * math.log(span / (2.0 * math.pi * turns)) / math.log(base)
        lo, hi = max(math.floor(where(32.0)), 0), min(math.ceil(where(1.0)), 2 * n - 1)
        r = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f * (1.0 - r) + f / factor * r, 0.1 * math.log(factor) + 1.0
    if scaling == "bands":  # whole above four turns over the old span, divided below one
        r = np.clip((span * f / (2.0 * math.pi) - 1.0) / 3.0, 0.0, 1.0)
        return f * r + f / factor * (1.0 - r), 1.0
    return f, 1.0


def _ints(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def _pool(case, g, seqs, spans):
    """A page pool that holds `spans` tokens of each sequence, its pages in no order, and its table."""
    page, H, D, block = case["page"], case["H"], case["D"], case["block"]
    pages = [-(-int(n) // page) for n in spans]
    total, width = sum(pages) + 1, max(max(pages), 1)
    order = torch.randperm(total, generator=g, device=DEV).int()
    at = np.zeros((seqs, width), dtype=np.int64)  # unused entries name the first page of the order
    first = 0
    for s, n in enumerate(pages):
        at[s, :n] = np.arange(first, first + n)
        first += n
    s = dict(table=order[torch.as_tensor(at, device=DEV)].contiguous())
    for name in ("k", "v"):
        x = torch.randn(total, H, page, D, generator=g, device=DEV, dtype=torch.float16)
        if case["fmt"] == "i8":
            s[name] = (x * 36.0).round().clamp(-127.0, 127.0).to(torch.int8).view(torch.uint8)
            d = (2.4 + 2.2 * torch.rand(total, H, page // block, generator=g, device=DEV)) / 127.0
            s[name + "_scale"] = (d * 4096.0 * 8.0).round() / (4096.0 * 8.0)  # 12 bits at most
        else:
            s[name] = (x * 100.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
            s[name + "_scale"] = torch.where(torch.rand(total, H, page // block, generator=g, device=DEV) < 0.7, 2.0 ** -7,
                                             2.0 ** -8)
    return s


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 29)
    op, t = case["op"], TYPES[case["type"]]
    if op == "rope":
        far = case["far"]
        start = torch.randint(0, max(1, far - case["T"]), (1,), generator=g, device=DEV)
        pos = (start + torch.arange(case["T"], device=DEV)) % far if case["T"] > 256 else \
            torch.randint(0, far, (case["T"],), generator=g, device=DEV)
        s = dict(x=torch.randn(case["T"], case["H"], case["D"], generator=g, device=DEV).to(t), pos=pos.int())
        f, s["magnitude"] = _freqs(case, case["rot"] // 2)
        s["freqs"] = torch.as_tensor(f, device=DEV)
        s["out"] = torch.empty_like(s["x"])
        return s
    lengths, H, D = _lengths(case), case["H"], case["D"]
    if op == "attend":
        s = _pool(case, g, case["seqs"], lengths)
        T, per = case["seqs"] * case["per"], case["per"]
        # attention that looks at some keys more than at others; one channel is an outlier
        q = torch.randn(T + case["pad"], case["Hq"], D, generator=g, device=DEV) * 2.0
        q[:, :, 3] *= 4.0
        s["q"] = q.to(t)
        seq, step = np.arange(T) // per, np.arange(T) % per
        s["seq"] = _ints(np.concatenate((seq, np.full(case["pad"], -1))))
        s["pos"] = _ints(np.concatenate((lengths[seq] - per + step, np.zeros(case["pad"], dtype=np.int64))))
        s["out"] = torch.empty_like(s["q"])
        return s
    news, block = _news(case), case["block"]
    s = _pool(case, g, case["seqs"], lengths + news)
    seq = np.repeat(np.arange(case["seqs"]), news)
    pos = np.concatenate([np.arange(a, a + n) for a, n in zip(lengths, news)])
    start = lengths // block * block  # what is read back: every token of the blocks that are written to
    back = [np.arange(a, b + n) for a, b, n in zip(start, lengths, news)]
    s.update(seq=_ints(seq), pos=_ints(pos), back_seq=_ints(np.repeat(np.arange(case["seqs"]), [len(b) for b in back])),
             back_pos=_ints(np.concatenate(back)), before=_ints(lengths))
    T = case["new"]
    for name, heads in (("new_k", H), ("new_v", H), ("q", case["Hq"])):
        x = torch.randn(T, heads, D, generator=g, device=DEV)
        s[name] = (x * (0.5 + torch.rand(T, 1, 1, generator=g, device=DEV))).to(t)
    f, s["magnitude"] = _freqs(case, D // 2)
    s["freqs"] = torch.as_tensor(f, device=DEV)
    s["q_out"] = torch.empty_like(s["q"])
    B = len(s["back_pos"])
    s["back_k"], s["back_v"] = (torch.empty(B, H, D, dtype=t, device=DEV) for _ in range(2))
    return s


def prepare(case, seed):
    """The buffers of a decode loop, its page pool and rotation table, and the step graph that it keeps over them."""
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    from decode_gemv_epilogue_gb300 import gemvfuse as gf

    typ = dict(f32=gf.F32, f16=gf.F16)[case["type"]]
    layout = dict(halves=gf.ROPE_HALVES, pairs=gf.ROPE_PAIRS)
    if case["op"] == "rope" or (case["op"] == "store" and case["rope"] != "none"):
        n = case.get("rot", case["D"])
        kind = dict(plain=gf.ROPE_PLAIN, linear=gf.ROPE_LINEAR, ramp=gf.ROPE_RAMP, bands=gf.ROPE_BANDS)[
            case.get("scaling", "plain")]
        s["rope"] = torch.empty(gf.rope_table_bytes(n), dtype=torch.uint8, device=DEV)
        gf.rope_table(s["rope"], n, base=case.get("base", 10000.0), kind=kind, factor=case.get("factor", 1.0), span=8192,
                      fast=4.0 if case.get("scaling") == "bands" else 32.0, slow=1.0)
    if case["op"] == "rope":
        s["graph"] = gf.Graph([gf.prepare_rope(s["x"], case["T"], case["H"], case["D"], s["pos"], s["rope"], s["out"],
                                               n_rot=case["rot"], layout=layout[case["layout"]], type=typ)])
        return s
    fmt = dict(i8=gf.CACHE_I8, e4m3=gf.CACHE_E4M3)[case["fmt"]]
    cache = gf.Cache(s["k"], s["v"], s["k_scale"], s["v_scale"], fmt, s["k"].shape[0], case["H"], case["page"], case["D"],
                     case["block"], s["table"], case["seqs"], s["table"].shape[1])
    if case["op"] == "store":
        turned = {} if case["rope"] == "none" else dict(rope=s["rope"], n_rot=case["D"], layout=layout[case["rope"]], q=s["q"],
                                                        q_heads=case["Hq"], q_dst=s["q_out"])
        calls = [gf.prepare_cache_store(cache, s["new_k"], s["new_v"], case["new"], s["seq"], s["pos"], type=typ, **turned),
                 gf.prepare_cache_load(cache, len(s["back_pos"]), s["back_seq"], s["back_pos"], s["back_k"], s["back_v"],
                                       type=typ, pdl=True)]
    else:
        T = case["seqs"] * case["per"] + case["pad"]
        s["workspace"] = torch.empty(gf.attend_workspace(T, case["Hq"], case["H"], case["D"], case["per"]), dtype=torch.uint8,
                                     device=DEV)
        calls = [gf.prepare_attend(cache, s["q"], T, case["Hq"], s["seq"], s["pos"], s["out"], s["workspace"], type=typ,
                                   window=case["window"], run=case["per"])]
    s["graph"] = gf.Graph(calls)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if own:
        state["graph"].launch()
        return _returned(case, state)
    return {"rope": _rope, "store": _store, "attend": _attend}[case["op"]](case, state)


def _returned(case, s):
    if case["op"] != "store":
        return s["out"]
    r = dict(k=s["back_k"], v=s["back_v"])
    return r if case["rope"] == "none" else dict(r, q=s["q_out"])


def _turn(x, pos, freqs, magnitude, layout):
    """x [T, H, D] in 32 bits, its first 2 len(freqs) elements of each head rotated."""
    n = len(freqs)
    angle = pos.double()[:, None] * freqs  # in 64 bits: far positions
    c, s = ((f(angle) * magnitude).float()[:, None, :] for f in (torch.cos, torch.sin))
    r = x[..., :2 * n]
    a, b = (r[..., 0::2], r[..., 1::2]) if layout == "pairs" else (r[..., :n], r[..., n:])
    u, v = a * c - b * s, a * s + b * c
    r = torch.stack((u, v), -1).flatten(-2) if layout == "pairs" else torch.cat((u, v), -1)
    return torch.cat((r, x[..., 2 * n:]), -1)


def _rope(case, s):
    return _turn(s["x"].float(), s["pos"], s["freqs"], s["magnitude"], case["layout"]).to(s["x"].dtype)


def _values(fmt, codes):
    return codes.view(torch.int8).float() if fmt == "i8" else codes.view(torch.float8_e4m3fn).float()


def _power(e):
    """2^e in 64 bits, from its bits: exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _scale_for(fmt, top):
    """The least scale that the format allows for values up to `top`."""
    top = top.double()
    m, e = torch.frexp(top / torch.full_like(top, MOST[fmt]))  # (a number's reciprocal would be rounded first)
    if fmt == "i8":
        d = torch.ceil(m * 4096.0) / 4096.0 * _power(e)
    else:
        d = _power(torch.where(m > 0.5, e, e - 1))
    return d.clamp(SMALLEST, LARGEST[fmt])


def _rounded(fmt, y):
    """y, in 64 bits, rounded to the format's codes, ties to even."""
    y = y.clamp(-MOST[fmt], MOST[fmt])
    if fmt == "i8":
        return y.round()
    step = _power(torch.frexp(y)[1].clamp_min(-5) - 4)
    return (y / step).round() * step


def _store(case, s):
    fmt, block, page = case["fmt"], case["block"], case["page"]
    seq, pos, bseq, bpos = (s[n].long() for n in ("seq", "pos", "back_seq", "back_pos"))
    before = s["before"].long()
    most = s["table"].shape[1] * page // block
    keys, of_new = torch.unique(seq * most + pos // block, return_inverse=True)  # the blocks that are written to
    of_back = torch.searchsorted(keys, bseq * most + bpos // block)
    kseq, kblk = keys // most, keys % most
    kpage = s["table"].long()[kseq, kblk * block // page]
    started = (before[kseq] > kblk * block)[:, None]
    fresh = bpos >= before[bseq]
    nth = torch.where(fresh, torch.cumsum(fresh, 0) - 1, 0)  # the new token that is read back
    bpage = s["table"].long()[bseq, bpos // page]
    out = {}
    for name in ("k", "v"):
        x = s["new_" + name].float()
        if name == "k" and case["rope"] != "none":
            x = _turn(x, s["pos"], s["freqs"], s["magnitude"], case["rope"])
        top = torch.zeros(len(keys), case["H"], device=DEV)
        top = top.scatter_reduce(0, of_new[:, None].expand(-1, case["H"]), x.abs().amax(2), "amax")
        old = torch.where(started, s[name + "_scale"][kpage, :, kblk % (page // block)].double(), 0.0)
        d = torch.maximum(_scale_for(fmt, top), old)
        new = _rounded(fmt, x.double() / d[of_new][..., None])
        kept = _values(fmt, s[name][bpage, :, bpos % page]).double()
        kept = _rounded(fmt, kept * (old / d)[of_back][..., None]) if fmt == "e4m3" else \
            _rounded(fmt, kept * old[of_back][..., None] / d[of_back][..., None])
        out[name] = (torch.where(fresh[:, None, None], new[nth], kept) * d[of_back][..., None]).to(s["new_k"].dtype)
    if case["rope"] != "none":
        out["q"] = _turn(s["q"].float(), s["pos"], s["freqs"], s["magnitude"], case["rope"]).to(s["q"].dtype)
    return out


def _attend(case, s):
    S, per, H, D, page = case["seqs"], case["per"], case["H"], case["D"], case["page"]
    table = s["table"].long()

    def whole(name):
        x = _values(case["fmt"], s[name][table]) * s[name + "_scale"][table].repeat_interleave(case["block"], -1)[..., None]
        return x.transpose(1, 2).reshape(S, H, -1, D)

    pos = s["pos"][:S * per].view(S, per).long()
    q = s["q"][:S * per].float().view(S, per, H, -1, D).permute(0, 2, 1, 3, 4).reshape(S, H, -1, D)
    a = (q @ whole("k").transpose(2, 3)).view(S, H, per, -1, table.shape[1] * page) * D ** -0.5
    j = torch.arange(a.shape[-1], device=a.device)
    seen = j <= pos[..., None]
    if case["window"]:
        seen = seen & (j > pos[..., None] - case["window"])
    a = torch.where(seen[:, None, :, None], a, float("-inf"))
    a = torch.exp(a - a.amax(-1, keepdim=True))
    z = a.sum(-1)
    o = (a.flatten(2, 3) @ whole("v")).view(S, H, per, -1, D) / z[..., None]
    o = o.permute(0, 2, 1, 3, 4).reshape(S * per, case["Hq"], D)
    return torch.cat((o, torch.zeros(case["pad"], case["Hq"], D, device=o.device))).to(s["q"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    size, D, H = (4 if case["type"] == "f32" else 2), case["D"], case["H"]
    if case["op"] == "rope":
        n = case["T"] * H * D
        return {"bytes": 2 * n * size + case["T"] * 4, "flops": 3 * case["T"] * H * case["rot"]}
    lengths = _lengths(case)
    if case["op"] == "store":
        T, block = case["new"], case["block"]
        back = int(np.sum(lengths % block)) + T
        b = T * (2 * H + 2 * case["Hq"]) * D * size + 2 * T * H * D  # new rows read, queries turned, codes written
        b += 2 * back * H * D * (1 + size)  # read back
        return {"bytes": b + 2 * (T // block + case["seqs"]) * H * 4, "flops": 4 * T * H * D + 3 * T * (case["Hq"] + H) * D}
    per, w = case["per"], case["window"]
    seen = np.minimum(lengths, w + per - 1) if w else lengths
    T = case["seqs"] * per + case["pad"]
    b = 2 * int(seen.sum()) * H * D + 2 * int(seen.sum()) // case["block"] * H * 4 + 2 * T * case["Hq"] * D * size
    each = np.minimum(lengths, w) if w else lengths
    return {"bytes": b, "flops": 4 * int(each.sum()) * per * case["Hq"] * D}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        return _exact_turn(s["x"], s["pos"], s["freqs"], s["magnitude"], case["layout"])
    if case["op"] == "store":
        return _exact_store(case, s)
    return _exact_attend(case, s)


def _exact_turn(x, pos, freqs, magnitude, layout):
    """As products with complex numbers."""
    n = len(freqs)
    z = torch.polar(torch.full((len(pos), 1, n), magnitude, dtype=torch.float64, device=x.device),
                    (pos.double()[:, None] * freqs)[:, None, :])
    y = x.double()
    p = y[..., :2 * n].unflatten(-1, (n, 2) if layout == "pairs" else (2, n))
    p = p if layout == "pairs" else p.transpose(-1, -2)
    r = torch.view_as_real(torch.view_as_complex(p.contiguous()) * z)
    y[..., :2 * n] = (r if layout == "pairs" else r.transpose(-1, -2)).flatten(-2)
    return y


def _e4m3_table():
    """Every finite non-negative value of the format, ascending; its position is its code."""
    v = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return np.array(v[:127])


def _exact_codes(fmt, y):
    """The format's value next to y, ties to the even code."""
    if fmt == "i8":
        return np.clip(np.rint(y), -127, 127)
    t = _e4m3_table()
    a = np.minimum(np.abs(y), 448.0)
    hi = np.minimum(np.searchsorted(t, a), len(t) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = t[hi] - a, a - t[lo]
    return np.copysign(np.where((up < down) | ((up == down) & (hi % 2 == 0)), t[hi], t[lo]), y)


def _exact_decode(fmt, raw):
    if fmt == "i8":
        return raw.view(np.int8).astype(np.float64)
    t = np.concatenate((_e4m3_table(), [np.nan]))
    return np.where(raw >= 128, -1.0, 1.0) * t[raw & 127]


def _exact_store(case, s):
    fmt, block, page, H = case["fmt"], case["block"], case["page"], case["H"]
    table, before = s["table"].cpu().numpy(), s["before"].cpu().numpy()
    seq, pos = s["seq"].cpu().numpy(), s["pos"].cpu().numpy()
    k = s["new_k"]
    if case["rope"] != "none":
        k = _exact_turn(k, s["pos"], s["freqs"], s["magnitude"], case["rope"])
    groups = {}  # (sequence, block) -> its new tokens, in the order in which they are read back
    for t in range(len(seq)):
        groups.setdefault((seq[t], pos[t] // block), []).append(t)
    out = {}
    for name, x in (("k", k), ("v", s["new_v"])):
        x = x.double().cpu().numpy()
        codes, scales = s[name], s[name + "_scale"]
        pages = np.array([table[q, b * block // page] for q, b in groups])
        subs = np.array([b % (page // block) for _, b in groups])
        at = torch.as_tensor(pages, device=codes.device).long()
        lines = codes[at].cpu().numpy().reshape(len(groups), H, page // block, block, -1) if len(groups) < 300 else None
        olds = scales[at].cpu().numpy().astype(np.float64)
        rows = []
        for i, ((q, b), ts) in enumerate(groups.items()):
            kept = max(0, int(min(before[q], (b + 1) * block) - b * block))
            top = np.abs(x[ts]).max(axis=(0, 2))
            m, e = np.frexp(top / MOST[fmt])
            need = np.ldexp(np.ceil(m * 4096) / 4096, e) if fmt == "i8" else np.ldexp(1.0, np.where(m > 0.5, e, e - 1))
            need = np.clip(need, SMALLEST, LARGEST[fmt])
            d = np.maximum(need, olds[i, :, subs[i]]) if kept else need
            if kept:
                raw = lines[i] if lines is not None else codes[pages[i]].cpu().numpy().reshape(H, page // block, block, -1)
                c = _exact_decode(fmt, raw[:, subs[i], :kept])
                c = _exact_codes(fmt, c * olds[i, :, subs[i]][:, None, None] / d[:, None, None])
                rows.append((c * d[:, None, None]).transpose(1, 0, 2))
            rows.append(_exact_codes(fmt, x[ts] / d[None, :, None]) * d[None, :, None])
        out[name] = torch.from_numpy(np.concatenate(rows))
    if case["rope"] != "none":
        out["q"] = _exact_turn(s["q"], s["pos"], s["freqs"], s["magnitude"], case["rope"])
    return out


def _exact_attend(case, s):
    H, D, page, block = case["H"], case["D"], case["page"], case["block"]
    G, w = case["Hq"] // H, case["window"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    values = torch.as_tensor(_exact_decode(case["fmt"], np.arange(256, dtype=np.uint8)), device=DEV)
    seq, pos = s["seq"].tolist(), s["pos"].tolist()
    for t, (n, p) in enumerate(zip(seq, pos)):
        if n < 0:
            continue
        if t == 0 or seq[t - 1] != n:  # a sequence's keys and values, up to its last token's
            last = max(b for a, b in zip(seq, pos) if a == n)
            j = torch.arange(last + 1, device=DEV)
            at = s["table"][n].long()[j // page]
            k, v = (values[s[m][at, :, j % page].long()] * s[m + "_scale"][at, :, j % page // block].double()[..., None]
                    for m in ("k", "v"))
        lo = max(0, p + 1 - w) if w else 0
        q = s["q"][t].double().view(H, G, D)
        a = torch.einsum("hgd,jhd->hgj", q, k[lo:p + 1]) / math.sqrt(D)
        out[t] = torch.einsum("hgj,jhd->hgd", torch.softmax(a, -1), v[lo:p + 1]).reshape(H * G, D)
    return out
