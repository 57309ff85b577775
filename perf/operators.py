"""Measured cases of the operators whose weights are chosen per column: routing to experts
(gf_route), the chosen experts' gated feed-forward product (gemv_experts) and a shared projection
with low-rank adapters per column (gemv_lora).

`run` computes them from elementary torch operations where `own` is false, and through the
library where it is true.  Storage formats of weight matrices (rows of K elements):
  f32, f16 : plain;                    q8_0 : per 32 elements an f16 scale and 32 int8 codes;
  q4_0     : per 32 an f16 scale and 16 bytes, byte j holding elements j (low nibble) and j + 16;
  q4_k     : per 256 two f16 scales, 12 bytes of 6-bit scales and mins, 128 bytes of codes.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
FORMATS = ("f32", "f16", "q8_0", "q4_0", "q4_k")
BLOCK = {"f32": (1, 4), "f16": (1, 2), "q8_0": (32, 34), "q4_0": (32, 18), "q4_k": (256, 144)}
NEG_INF = float("-inf")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One token of one user through a router of 128 experts: latency only.
        dict(name="route_token", op="route", T=1, E=128, k=8, score="softmax", bias=False, groups=1, keep=1,
             norm=True, scale=1.0, masked=0.0),
        # A decode batch through a sigmoid router with a balancing bias and groups of experts.
        dict(name="route_batch_groups", op="route", T=61, E=256, k=8, score="sigmoid", bias=True, groups=8,
             keep=4, norm=True, scale=2.5, masked=0.0),
        # An odd number of tokens and experts, a quarter of the experts masked (not resident).
        dict(name="route_odd_masked", op="route", T=1023, E=60, k=4, score="softmax", bias=True, groups=1,
             keep=1, norm=False, scale=1.0, masked=0.25),
        # A long prompt, or many of them packed together.
        dict(name="route_prompt", op="route", T=16384, E=128, k=8, score="softmax", bias=False, groups=1, keep=1,
             norm=True, scale=1.0, masked=0.0),
        # One token through eight small experts in 4 bits: the single user's decode step.
        dict(name="experts_token_q4_k", op="experts", T=1, E=128, k=8, K=2048, M=768, fmt="q4_k", down="q4_k",
             add=True),
        # A few users; the expert width is no multiple of 256.
        dict(name="experts_few_q4_0", op="experts", T=7, E=64, k=6, K=2048, M=1408, fmt="q4_0", down="q4_0",
             add=False),
        # A small batch through 8-bit experts.
        dict(name="experts_batch_q8_0", op="experts", T=16, E=32, k=4, K=2048, M=1024, fmt="q8_0", down="q8_0",
             add=True),
        # Few large experts kept in f16, an odd batch.
        dict(name="experts_large_f16", op="experts", T=33, E=8, k=2, K=4096, M=14336, fmt="f16", down="f16",
             add=True),
        # The widest batch: every expert is read, about sixteen columns each.
        dict(name="experts_wide_q4_k", op="experts", T=256, E=128, k=8, K=2048, M=768, fmt="q4_k", down="q4_k",
             add=True),
        # One user with an adapter on a 4-bit projection.
        dict(name="lora_token_q4_0", op="lora", N=1, M=4096, K=4096, fmt="q4_0", n=8, r=16, afmt="f16", tail="none",
             bare=0),
        # Eight users with adapters of their own (one with none) on an f16 output projection.
        dict(name="lora_batch_f16", op="lora", N=8, M=4096, K=4096, fmt="f16", n=8, r=16, afmt="f16", tail="add",
             bare=1),
        # A wide batch, large adapters, the gate of a feed-forward layer.
        dict(name="lora_wide_q4_0", op="lora", N=64, M=14336, K=4096, fmt="q4_0", n=16, r=64, afmt="f16",
             tail="silu", bare=5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "experts", "lora"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        E = groups * _log_int(rng, max(2, 8 // groups), 256 // groups)
        keep = groups if groups == 1 else rng.randint(1, groups - 1)
        k = rng.randint(1, min(12, keep * (E // groups)))
        score = rng.choice(("softmax", "sigmoid"))
        T = _log_int(rng, 1, min(16384, 16384 * 128 // E))
        return dict(op="route", T=T, E=E, k=k, score=score, bias=groups > 1 or rng.random() < 0.5, groups=groups,
                    keep=keep, norm=rng.random() < 0.7, scale=rng.choice((1.0, 1.5, 2.5)),
                    masked=rng.choice((0.0, 0.0, 0.2)))
    if op == "experts":
        fmt = rng.choice(FORMATS)
        down = rng.choice((fmt, fmt, "q8_0" if fmt == "q4_k" else fmt))
        E = rng.choice((4, 8, 16, 32, 60, 64, 128))
        step = 256 if "q4_k" in (fmt, down) else 32
        K = step * _log_int(rng, 512 // step, 4096 // step)
        M = step * _log_int(rng, 256 // step, 4096 // step)
        while E * M * K > 8 * 4096 * 14336:
            E //= 2
        return dict(op="experts", T=_log_int(rng, 1, 256), E=E, k=rng.randint(1, min(8, E)), K=K, M=M, fmt=fmt,
                    down=down, add=rng.random() < 0.5)
    fmt = rng.choice(FORMATS)
    step = 256 if fmt == "q4_k" else 32
    N = _log_int(rng, 1, 64)
    return dict(op="lora", N=N, M=_log_int(rng, 256, 14336), K=step * _log_int(rng, 512 // step, 4096 // step), fmt=fmt,
                n=_log_int(rng, 1, 16), r=rng.choice((4, 8, 16, 24, 32, 64)), afmt=rng.choice(("f16", "f16", "f32")),
                tail=rng.choice(("none", "add", "silu", "sigmoid")), bare=rng.randint(0, N - 1) if N > 1 else 0)


# ------------------------------------------------------------------ inputs

def _weights(g, fmt, rows, K, std):
    """rows x K random weights of about the given spread, as the bytes of the format."""
    if fmt == "f32":
        return torch.randn(rows, K, generator=g, device=DEV) * std
    if fmt == "f16":
        return torch.randn(rows, K, generator=g, device=DEV, dtype=torch.float16) * std
    n, size = BLOCK[fmt]
    raw = torch.randint(0, 256, (rows, K // n, size), generator=g, device=DEV, dtype=torch.uint8)
    u = 0.5 + torch.rand(rows, K // n, 1, generator=g, device=DEV)
    spread = {"q8_0": 74.0, "q4_0": 4.7, "q4_k": 250.0}[fmt]  # of the codes (times 6-bit scales)
    d = (u * (std / spread)).half()
    raw[:, :, 0:2] = d.view(torch.uint8)
    if fmt == "q4_k":  # the mins centre the codes 0..15
        raw[:, :, 2:4] = (d * 7.5).view(torch.uint8)
    return raw.view(rows, -1)


def _logits(g, T, E, masked):
    l = torch.randn(T, E, generator=g, device=DEV) * 1.5
    if masked:
        l = l.masked_fill(torch.rand(T, E, generator=g, device=DEV) < masked, NEG_INF)
    return l


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        s = dict(logits=_logits(g, T, E, case["masked"]), bias=None)
        if case["bias"]:
            s["bias"] = torch.randn(E, generator=g, device=DEV) * 0.05
        s["ids"] = torch.empty(T, case["k"], dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty(T, case["k"], device=DEV)
        return s
    if case["op"] == "experts":
        T, E, k, K, M = case["T"], case["E"], case["k"], case["K"], case["M"]
        p, i = torch.softmax(_logits(g, T, E, 0.0), 1).topk(k, dim=1)
        return dict(gate=_weights(g, case["fmt"], E * M, K, K ** -0.5), up=_weights(g, case["fmt"], E * M, K, K ** -0.5),
                    down=_weights(g, case["down"], E * K, M, M ** -0.5),
                    x=torch.randn(T, K, generator=g, device=DEV), ids=i.int().contiguous(),
                    weights=(p / p.sum(1, keepdim=True)).contiguous(),
                    aux=torch.randn(T, K, generator=g, device=DEV) if case["add"] else None,
                    dst=torch.empty(T, K, device=DEV))
    N, M, K, n, r = case["N"], case["M"], case["K"], case["n"], case["r"]
    ids = torch.randint(0, n, (N,), generator=g, device=DEV, dtype=torch.int32)
    ids[torch.randperm(N, generator=g, device=DEV)[:case["bare"]]] = -1
    at = torch.float16 if case["afmt"] == "f16" else torch.float32
    return dict(W=_weights(g, case["fmt"], M, K, K ** -0.5),
                A=(torch.randn(n, r, K, generator=g, device=DEV) * K ** -0.5).to(at),
                B=(torch.randn(n, M, r, generator=g, device=DEV) * r ** -0.5).to(at),
                scales=0.25 + torch.rand(n, generator=g, device=DEV), ids=ids,
                x=torch.randn(N, K, generator=g, device=DEV),
                aux=torch.randn(N, M, generator=g, device=DEV) if case["tail"] == "add" else None,
                dst=torch.empty(N, M, device=DEV))


def prepare(case, seed):
    """The buffers of a decode loop, and the step graph that it keeps over them."""
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    from decode_gemv_epilogue_gb300 import gemvfuse as gf

    wt = dict(f32=gf.F32, f16=gf.F16, q8_0=gf.Q8_0, q4_0=gf.Q4_0, q4_k=gf.Q4_K)
    if case["op"] == "route":
        call = gf.prepare_route(s["logits"], case["T"], case["E"], case["k"], s["ids"], s["weights"],
                                score=gf.SCORE_SIGMOID if case["score"] == "sigmoid" else gf.SCORE_SOFTMAX,
                                bias=s["bias"], n_group=case["groups"], topk_group=case["keep"], group_top=2,
                                norm=case["norm"], scale=case["scale"])
    elif case["op"] == "experts":
        T, E, k, K, M = case["T"], case["E"], case["k"], case["K"], case["M"]
        a, b = wt[case["fmt"]], wt[case["down"]]
        s["workspace"] = torch.empty(gf.experts_workspace(E, T, k, M, K), dtype=torch.uint8, device=DEV)
        call = gf.prepare_experts(s["gate"], s["up"], a, s["down"], b, E, s["x"], M, K, s["ids"], s["weights"], T, k,
                                  s["aux"], s["dst"], s["workspace"])
    else:
        N, M, K, n, r = case["N"], case["M"], case["K"], case["n"], case["r"]
        tail = dict(none=gf.EPI_NONE, add=gf.EPI_ADD, silu=gf.EPI_SILU, sigmoid=gf.EPI_SIGMOID)[case["tail"]]
        s["workspace"] = torch.empty(gf.lora_workspace(N, M, K, r, n), dtype=torch.uint8, device=DEV)
        call = gf.prepare_lora(s["W"], wt[case["fmt"]], s["x"], M, K, tail, s["aux"], s["dst"], s["A"], s["B"],
                               wt[case["afmt"]], n, r, s["ids"], s["scales"], s["workspace"], ncols=N)
    s["graph"] = gf.Graph([call])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if own:
        state["graph"].launch()
        return (state["ids"], state["weights"]) if case["op"] == "route" else state["dst"]
    return {"route": _route, "experts": _experts, "lora": _lora}[case["op"]](case, state)


def _route(case, s):
    l = s["logits"].double()  # in 64 bits: which of two near experts is taken
    live = l > NEG_INF
    if case["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.max(1, keepdim=True).values)
        p = e / e.sum(1, keepdim=True)
    key = p if s["bias"] is None else p + s["bias"].double()
    key = torch.where(live, key, NEG_INF)
    G, E = case["groups"], case["E"]
    if G > 1:
        top = key.view(-1, G, E // G).sort(dim=2, descending=True).values[:, :, :2]
        g = torch.where(top > NEG_INF, top, 0.0).sum(2)
        g = torch.where(top[:, :, 0] > NEG_INF, g, NEG_INF)
        order = g.sort(dim=1, descending=True, stable=True).indices[:, :case["keep"]]
        kept = torch.zeros_like(g).scatter(1, order, 1.0) > 0
        key = torch.where(kept.repeat_interleave(E // G, 1), key, NEG_INF)
    key, i = key.sort(dim=1, descending=True, stable=True)
    key, i = key[:, :case["k"]], i[:, :case["k"]]
    w = torch.where(key > NEG_INF, p.gather(1, i), 0.0)
    if case["norm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    return torch.where(key > NEG_INF, i, -1).int(), (w * case["scale"]).float()


def _half(b):
    return b.contiguous().view(torch.float16).float()


def _values(fmt, raw):
    """[..., row bytes] -> [..., K] in 32 bits; every stored value is exact in them."""
    if fmt in ("f32", "f16"):
        return raw.float()
    n, size = BLOCK[fmt]
    b = raw.unflatten(-1, (-1, size))
    if fmt == "q8_0":
        v = _half(b[..., 0:2]) * b[..., 2:].contiguous().view(torch.int8).float()
    elif fmt == "q4_0":
        c = b[..., 2:]
        v = _half(b[..., 0:2]) * (torch.cat((c & 15, c >> 4), -1).float() - 8.0)
    else:
        a, m, h = b[..., 4:8], b[..., 8:12], b[..., 12:16]
        sc = torch.cat((a & 63, (h & 15) | ((a >> 6) << 4)), -1).float()
        mn = torch.cat((m & 63, (h >> 4) | ((m >> 6) << 4)), -1).float()
        c = b[..., 16:].unflatten(-1, (4, 32))
        q = torch.stack((c & 15, c >> 4), -2).flatten(-3, -2).float()  # [..., 8, 32]
        v = ((_half(b[..., 0:2]) * sc).unsqueeze(-1) * q - (_half(b[..., 2:4]) * mn).unsqueeze(-1)).flatten(-2)
    return v.flatten(-2)


def _silu(y):
    return y / (1.0 + torch.exp(-y))


def _experts(case, s):
    T, E, k, K, M = case["T"], case["E"], case["k"], case["K"], case["M"]
    x, i = s["x"], s["ids"].long()
    gate, up, down = s["gate"].view(E, M, -1), s["up"].view(E, M, -1), s["down"].view(E, K, -1)
    if T * k < E:  # few slots: their experts' weights side by side
        i = i.flatten()
        xs = x.repeat_interleave(k, 0).unsqueeze(2)
        h = _silu(_values(case["fmt"], gate[i]) @ xs) * (_values(case["fmt"], up[i]) @ xs)
        y = (_values(case["down"], down[i]) @ h).view(T, k, K)
        y = (y * s["weights"].unsqueeze(2)).sum(1)
    else:  # every expert on every token, weighted by zero where it is not chosen
        h = _silu(x @ _values(case["fmt"], gate).transpose(1, 2)) * (x @ _values(case["fmt"], up).transpose(1, 2))
        c = torch.zeros(T, E, device=x.device).scatter_add(1, i, s["weights"])
        y = ((h * c.t().unsqueeze(2)) @ _values(case["down"], down).transpose(1, 2)).sum(0)
    return y if s["aux"] is None else y + s["aux"]


def _lora(case, s):
    x, i = s["x"], s["ids"].long()
    j = i.clamp_min(0)
    v = (s["A"].float()[j] @ x.unsqueeze(2)) * torch.where(i >= 0, s["scales"][j], 0.0)[:, None, None]
    y = x @ _values(case["fmt"], s["W"]).t() + (s["B"].float()[j] @ v).squeeze(2)
    if case["tail"] == "add":
        return y + s["aux"]
    if case["tail"] == "silu":
        return _silu(y)
    return 1.0 / (1.0 + torch.exp(-y)) if case["tail"] == "sigmoid" else y


# ------------------------------------------------------------------ what a pass cannot do without

def _matrix(fmt, rows, K):
    n, size = BLOCK[fmt]
    return rows * (K // n) * size


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * 4 + T * k * 8 + (E * 4 if case["bias"] else 0), "flops": T * E * 4}
    if case["op"] == "experts":
        T, E, k, K, M = case["T"], case["E"], case["k"], case["K"], case["M"]
        read = E * (1.0 - (1.0 - k / E) ** T)  # experts that at least one token takes, on average
        b = read * (2 * _matrix(case["fmt"], M, K) + _matrix(case["down"], K, M))
        return {"bytes": b + T * K * 4 * (3 if case["add"] else 2) + T * k * 8, "flops": 2 * T * k * 3 * M * K}
    N, M, K, n, r = case["N"], case["M"], case["K"], case["n"], case["r"]
    used = N - case["bare"]
    read = n * (1.0 - (1.0 - 1.0 / n) ** used)
    b = _matrix(case["fmt"], M, K) + read * r * (M + K) * (2 if case["afmt"] == "f16" else 4)
    return {"bytes": b + N * K * 4 + N * M * 4 * (2 if case["tail"] == "add" else 1) + N * 4,
            "flops": 2 * N * M * K + 2 * used * r * (M + K)}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "experts":
        return _exact_experts(case, s)
    y = s["x"].double() @ _decode(case["fmt"], s["W"], case["K"]).t()
    for c, a in enumerate(s["ids"].tolist()):
        if a >= 0:
            y[c] += float(s["scales"][a]) * (s["B"][a].double() @ (s["A"][a].double() @ s["x"][c].double()))
    if case["tail"] == "add":
        y += s["aux"].double()
    elif case["tail"] != "none":
        y = torch.sigmoid(y) * (y if case["tail"] == "silu" else 1.0)
    return y


def _decode(fmt, raw, K):
    """Element by element: where the scale and the code of element e of a row lie."""
    if fmt in ("f32", "f16"):
        return raw.double()
    n, size = BLOCK[fmt]
    e = torch.arange(K, device=raw.device)
    base, o = e // n * size, e % n

    def half_at(p):
        return (raw[:, p].int() | (raw[:, p + 1].int() << 8)).to(torch.int16).view(torch.float16).double()

    if fmt == "q8_0":
        c = raw[:, base + 2 + o].double()
        return half_at(base) * torch.where(c > 127, c - 256, c)
    if fmt == "q4_0":
        c = raw[:, base + 2 + o % 16].int()
        return half_at(base) * (torch.where(o < 16, c % 16, c // 16) - 8).double()
    j = o // 32
    t = base + 4 + j % 4
    lo, mid, hi = raw[:, t].int(), raw[:, t + 4].int(), raw[:, t + 8].int()
    sc = torch.where(j < 4, lo % 64, hi % 16 + lo // 64 * 16)
    mn = torch.where(j < 4, mid % 64, hi // 16 + mid // 64 * 16)
    c = raw[:, base + 16 + o // 64 * 32 + o % 32].int()
    q = torch.where(j % 2 == 0, c % 16, c // 16)
    return half_at(base) * (sc * q).double() - half_at(base + 2) * mn.double()


def _exact_route(case, s):
    l = s["logits"].double().cpu().numpy()
    b = None if s["bias"] is None else s["bias"].double().cpu().numpy()
    T, E, G, k = case["T"], case["E"], case["groups"], case["k"]
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.exp(-np.logaddexp(0.0, -l)) if case["score"] == "sigmoid" else \
            np.exp(l - np.logaddexp.reduce(l, axis=1, keepdims=True))
    ids, w = np.full((T, k), -1, dtype=np.int32), np.zeros((T, k))
    for t in range(T):
        key = np.where(np.isneginf(l[t]), -np.inf, p[t] + (0.0 if b is None else b))
        if G > 1:
            best = [np.sort(q[q > -np.inf])[::-1][:2] for q in key.reshape(G, -1)]
            rank = sorted(range(G), key=lambda g: (-(best[g].sum() if len(best[g]) else -np.inf), g))
            for g in rank[case["keep"]:]:
                key[g * (E // G):(g + 1) * (E // G)] = -np.inf
        order = [e for e in np.argsort(-key, kind="stable")[:k] if key[e] > -np.inf]
        ids[t, :len(order)] = order
        w[t, :len(order)] = p[t, order]
        if case["norm"] and order:
            w[t] /= w[t].sum()
    return torch.from_numpy(ids), torch.from_numpy(w * case["scale"])


def _exact_experts(case, s):
    E, K, M = case["E"], case["K"], case["M"]
    x = s["x"].double()
    y = torch.zeros_like(x) if s["aux"] is None else s["aux"].double()
    for e in range(E):
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        at, to = slice(e * M, (e + 1) * M), slice(e * K, (e + 1) * K)
        g = x[t] @ _decode(case["fmt"], s["gate"][at], K).t()
        u = x[t] @ _decode(case["fmt"], s["up"][at], K).t()
        h = g * torch.sigmoid(g) * u
        y.index_add_(0, t, (h @ _decode(case["down"], s["down"][to], M).t()) * s["weights"][t, j].double()[:, None])
    return y
