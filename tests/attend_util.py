"""Helpers of the tests of rotary positions, the 8-bit cache and attention: random caches on both sides and
the tolerances, derived from the kernels' roundings (u = 2^-24 in 32 bits)."""

import numpy as np

from oracle import attend as oatt

U = 2.0 ** -24
HALF = 2.0 ** -11  # half a step of binary16


def cache_arrays(rng, fmt, n_pages, heads, page, dim, block, table, codes="random"):
    """An oracle cache with random codes (every finite one) and scales within a factor of eight."""
    c = dict(fmt=fmt, block=block, table=np.asarray(table, dtype=np.int32))
    for name in "kv":
        if codes == "random":
            x = rng.integers(0, 256, (n_pages, heads, page, dim), dtype=np.uint8)
            x[x == (0x80 if fmt == "i8" else 0x7f)] = 1
            x[x == (0x80 if fmt == "i8" else 0xff)] = 2
        else:
            x = np.zeros((n_pages, heads, page, dim), dtype=np.uint8)
        c[name] = x
        shape = (n_pages, heads, page // block)
        if fmt == "i8":  # values about 1
            s = rng.integers(1024, 4096, shape) * 2.0 ** -17
        else:
            s = 2.0 ** rng.integers(-8, -5, shape)
        c[name + "_scale"] = s.astype(np.float32)
    return c


def shuffled_table(rng, lengths, page, spare=1):
    """A table whose rows hold `lengths` tokens in pages of no order; (table, pages)."""
    need = [max(1, -(-int(n) // page)) for n in lengths]
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(need), max(need)), -1, dtype=np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


class DeviceCache:
    """The arrays of an oracle cache on the GPU and the library's struct over them."""

    def __init__(self, lib, c, device="cuda"):
        import torch
        self.t = {k: torch.from_numpy(c[k].copy()).to(device) for k in ("k", "v", "k_scale", "v_scale", "table")}
        n_pages, heads, page, dim = c["k"].shape
        self.cache = lib.Cache(self.t["k"], self.t["v"], self.t["k_scale"], self.t["v_scale"],
                               lib.CACHE_I8 if c["fmt"] == "i8" else lib.CACHE_E4M3, n_pages, heads, page, dim, c["block"],
                               self.t["table"], c["table"].shape[0], c["table"].shape[1])

    def host(self, name):
        return self.t[name].cpu().numpy()


def attend_bounds(c, want, lse, mass, spread, keys, f16):
    """Tolerances of (out, lse) element by element.
    A score: q in two parts 2^-22; dim / 16 matrix instructions, whose sums are cut, 2^-22 of the absolute
    sum each; hi + lo and three products, 2^-24 each.  A weight: both its own score's error and the
    largest's, the exponential's argument (its size in units) and two units of the exponential.  The sums: the
    weights' parts and the matrix unit 2^-20; a rounding for every chunk of 16 keys, for the chunk's scaling, and
    for up to 300 joined parts."""
    D = c["k"].shape[3]
    ds = spread * (2.0 ** -22 * (1 + D / 16) + 4 * U)
    rel = 2 * ds + 4 * U * (1 + spread) + 2.0 ** -20 + (keys / 16 + 300) * 4 * U
    b = mass * rel[..., None] + 1e-30
    if f16:
        b = b + np.abs(want) * HALF + 2.0 ** -25
    bl = ds + 4 * U * (1 + spread) + (keys / 16 + 300) * 4 * U + 4 * U * np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return b, bl


def norm_error(got, want):
    return float(np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-300))


# q and the weights as pairs of binary16 leave some 2^-22 of the result; without the low parts 2^-12 would be
# left, and with parts of bfloat16 2^-17 of a score times its size.
NORM_TOL = 2.0 ** -17


def exact_parts(x, n):
    """x as the sum of n binary16 parts under a power of two a row (last axis)."""
    top = np.abs(x).max(axis=-1, keepdims=True)
    f = 2.0 ** (14 - np.floor(np.log2(np.where(top > 0, top, 1.0))))
    y = np.zeros_like(x)
    for _ in range(n):
        y = y + (x * f - y).astype(np.float16).astype(np.float64)
    return y / f


def positions(lengths, per):
    """seq, pos of `per` tokens at the end of each sequence."""
    seq = np.repeat(np.arange(len(lengths)), per).astype(np.int32)
    pos = np.concatenate([np.arange(n - per, n) for n in lengths]).astype(np.int32)
    return seq, pos


def dequantised(c, seq, pos):
    return oatt.load(c, seq, pos)
