"""Oracle of a decode step's attention (fp64): rotary positions, the 8-bit cache, attention over it.
Test infrastructure only.  The formulas are the ones in include/gemvfuse.h (gf_rope, gf_cache_store,
gf_cache_load, gf_attend); the pages have no counterpart.  Written out token by token.

A cache is a dict of numpy arrays: k, v uint8 [n_pages, heads, page, dim], k_scale, v_scale float32
[n_pages, heads, page // block], table int32 [n_seqs, table_ld]; fmt "i8" or "e4m3", block.
"""

import math

import numpy as np

LARGEST_CODE = {"i8": 127.0, "e4m3": 448.0}
SCALE_MIN, SCALE_MAX = 2.0 ** -112, {"i8": 2.0 ** 121, "e4m3": 2.0 ** 119}


# ------------------------------------------------------------------ rotary positions

def freqs(n_rot, base=10000.0, kind="plain", factor=1.0, span=0, fast=32.0, slow=1.0, divisors=None):
    """float64 [n_rot / 2], radians a position."""
    n = n_rot // 2
    out = np.zeros(n)
    for i in range(n):
        f = base ** (-2.0 * i / n_rot)
        if kind == "linear":
            f = f / factor
        elif kind == "ramp":
            def x(turns):
                return n * math.log(span / (2.0 * math.pi * turns)) / math.log(base)
            lo = min(max(math.floor(x(fast)), 0), n_rot - 1)
            hi = min(max(math.ceil(x(slow)), 0), n_rot - 1)
            r = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = (1.0 - r) * f + r * f / factor
        elif kind == "bands":
            turns = span * f / (2.0 * math.pi)
            r = 1.0 - min(max((turns - slow) / (fast - slow), 0.0), 1.0)
            f = (1.0 - r) * f + r * f / factor
        out[i] = f if divisors is None else f / float(divisors[i])
    return out


def magnitude(kind="plain", factor=1.0, given=0.0):
    if given:
        return given
    return 0.1 * math.log(factor) + 1.0 if kind == "ramp" and factor > 1.0 else 1.0


def rope(x, pos, f, m=1.0, layout="halves"):
    """x [T, H, D] -> float64."""
    y = np.asarray(x, dtype=np.float64).copy()
    n = len(f)
    for t in range(y.shape[0]):
        for i in range(n):
            a, b = (i, n + i) if layout == "halves" else (2 * i, 2 * i + 1)
            ang = math.fmod(float(int(pos[t])) * f[i], 2.0 * math.pi)
            c, s = math.cos(ang) * m, math.sin(ang) * m
            u, v = y[t, :, a].copy(), y[t, :, b].copy()
            y[t, :, a] = u * c - v * s
            y[t, :, b] = u * s + v * c
    return y


# ------------------------------------------------------------------ the code formats

def e4m3_values():
    """The 256 values of the codes (NaN at 0x7f and 0xff)."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = np.nan if e == 15 and m == 7 else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        v[c] = -a if c >= 128 else a
    return v


E4M3 = e4m3_values()


def decode(fmt, codes):
    codes = np.asarray(codes, dtype=np.uint8)
    return codes.view(np.int8).astype(np.float64) if fmt == "i8" else E4M3[codes]


def encode(fmt, y):
    """The code next to each value of y (finite float64), ties to even; beyond the largest: the largest."""
    y = np.asarray(y, dtype=np.float64)
    if fmt == "i8":
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    t = E4M3[:127]
    a = np.minimum(np.abs(y), 448.0)
    hi = np.minimum(np.searchsorted(t, a), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = t[hi] - a, a - t[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (c + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def least_scale(fmt, top):
    """For values of magnitude up to `top` (finite)."""
    top = float(top)
    if top == 0.0:
        return SCALE_MIN
    m, e = math.frexp(top / LARGEST_CODE[fmt])  # top / 127 is no tie of 12 bits unless it is exact
    if fmt == "i8":
        d = math.ldexp(math.ceil(m * 4096.0) / 4096.0, e)
    else:
        d = math.ldexp(1.0, e if m > 0.5 else e - 1)
    return min(max(d, SCALE_MIN), SCALE_MAX[fmt])


# ------------------------------------------------------------------ the cache

def place(cache, seq, pos):
    """(page, slot) of a token, or None."""
    page, table = cache["k"].shape[2], cache["table"]
    if seq < 0 or seq >= table.shape[0] or pos < 0 or pos // page >= table.shape[1]:
        return None
    p = int(table[seq, pos // page])
    return (p, int(pos % page)) if 0 <= p < cache["k"].shape[0] else None


def store(cache, k, v, seq, pos):
    """In place.  k, v [T, heads, dim], the exact values to be stored."""
    fmt, block = cache["fmt"], cache["block"]
    runs = []  # neighbouring tokens of one block
    for t in range(len(pos)):
        if place(cache, int(seq[t]), int(pos[t])) is None:
            continue
        if runs and t > 0 and runs[-1][-1] == t - 1 and seq[t] == seq[t - 1] and pos[t] == pos[t - 1] + 1 and \
                pos[t] // block == pos[t - 1] // block:
            runs[-1].append(t)
        else:
            runs.append([t])
    for ts in runs:
        page, slot = place(cache, int(seq[ts[0]]), int(pos[ts[0]]))
        first = int(pos[ts[0]]) % block
        for name, x in (("k", k), ("v", v)):
            x = np.asarray(x, dtype=np.float64)
            for h in range(cache["k"].shape[1]):
                new = x[ts, h]
                codes, scales, b = cache[name][page, h], cache[name + "_scale"][page, h], slot // block
                old = float(scales[b])
                if not np.all(np.isfinite(new)) or (first > 0 and np.isnan(old)):
                    scales[b] = np.nan
                    codes[slot:slot + len(ts)] = 0
                    continue
                d = least_scale(fmt, np.abs(new).max())
                if first > 0:
                    if d > old:
                        kept = decode(fmt, codes[slot - first:slot])
                        codes[slot - first:slot] = encode(fmt, kept * old / d)
                    d = max(d, old)
                codes[slot:slot + len(ts)] = encode(fmt, new / d)
                scales[b] = d


def load(cache, seq, pos):
    """k, v float64 [T, heads, dim]; zeros where a token has no place."""
    T, (_, H, _, D) = len(pos), cache["k"].shape
    out = np.zeros((2, T, H, D))
    for t in range(T):
        at = place(cache, int(seq[t]), int(pos[t]))
        if at is None:
            continue
        for i, name in enumerate("kv"):
            with np.errstate(invalid="ignore"):
                out[i, t] = decode(cache["fmt"], cache[name][at[0], :, at[1]]) * \
                    cache[name + "_scale"][at[0], :, at[1] // cache["block"]].astype(np.float64)[:, None]
    return out[0], out[1]


# ------------------------------------------------------------------ attention

def seen(cache, seq, pos, window=0):
    """Positions whose keys a token sees."""
    if seq < 0 or seq >= cache["table"].shape[0] or pos < 0:
        return []
    lo = max(0, pos + 1 - window) if window else 0
    hi = min(pos + 1, cache["table"].shape[1] * cache["k"].shape[2])
    return [j for j in range(lo, hi) if place(cache, seq, j) is not None]


def attend(cache, q, seq, pos, scale=None, window=0):
    """out [T, Hq, D], lse [T, Hq] (float64), and per output the size that its error is measured by:
    `mass` = sum_j softmax_j |V_j|, `spread` [T, Hq] = max_j scale * sum_d |q_d K_jd|."""
    q = np.asarray(q, dtype=np.float64)
    T, Hq, D = q.shape
    H = cache["k"].shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros(q.shape), np.full((T, Hq), -np.inf)
    mass, spread = np.zeros(q.shape), np.zeros((T, Hq))
    held = {}
    for t in range(T):
        s, p = int(seq[t]), int(pos[t])
        js = seen(cache, s, p, window)
        if not js:
            continue
        if s not in held or len(held[s][0]) <= p:  # every key of the sequence up to its last token here
            last = max(int(pos[i]) for i in range(T) if int(seq[i]) == s)
            last = min(last, cache["table"].shape[1] * cache["k"].shape[2] - 1)
            held[s] = load(cache, np.full(last + 1, s), np.arange(last + 1))
        k, v = held[s][0][js], held[s][1][js]  # [n, H, D]
        for h in range(Hq):
            kv = h // (Hq // H)
            with np.errstate(invalid="ignore", over="ignore"):
                a = scale * (k[:, kv] @ q[t, h])
                m = a.max()
                e = np.exp(a - m)
                z = e.sum()
                out[t, h] = e @ v[:, kv] / z
                lse[t, h] = m + np.log(z)
                mass[t, h] = e @ np.abs(v[:, kv]) / z
                spread[t, h] = scale * (np.abs(k[:, kv]) @ np.abs(q[t, h])).max()
    return out, lse, mass, spread
