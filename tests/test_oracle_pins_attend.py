"""Pins for the oracle of rotary positions, the 8-bit cache and attention: worked values, closed forms,
invariants, and planted mistakes that a pin has to catch."""

import math

import numpy as np
import pytest

import attend_util as au
from oracle import attend as oatt


# ------------------------------------------------------------------ rotary positions

def test_freqs_plain_and_linear():
    f = oatt.freqs(8, base=10000.0)
    assert np.allclose(f, [1.0, 0.1, 0.01, 0.001], rtol=1e-14)
    assert np.allclose(oatt.freqs(8, kind="linear", factor=4.0), f / 4, rtol=1e-14)
    assert np.allclose(oatt.freqs(8, divisors=[1, 2, 4, 8]), f / [1, 2, 4, 8], rtol=1e-14)


def test_freqs_ramp_ends():
    plain, f = oatt.freqs(64), oatt.freqs(64, kind="ramp", factor=8.0, span=4096, fast=32.0, slow=1.0)
    turns = 4096 * plain / (2 * math.pi)
    assert np.array_equal(f[turns > 60], plain[turns > 60])           # fast pairs stay
    assert np.allclose(f[turns < 0.5], plain[turns < 0.5] / 8, rtol=1e-14)  # slow ones are stretched
    r = (plain - f) / (plain - plain / 8)
    assert np.all(np.diff(r) >= -1e-12) and np.allclose(np.diff(r[(r > 0.01) & (r < 0.99)]), np.diff(r[(r > 0.01) & (r < 0.99)])[0])
    assert oatt.magnitude("ramp", 8.0) == 0.1 * math.log(8.0) + 1.0 and oatt.magnitude("ramp", 0.5) == 1.0
    assert oatt.magnitude("bands", 8.0) == 1.0 and oatt.magnitude("plain", given=0.5) == 0.5


def test_freqs_bands_ends():
    plain, f = oatt.freqs(64, base=500000.0), oatt.freqs(64, base=500000.0, kind="bands", factor=8.0, span=8192, fast=4.0, slow=1.0)
    turns = 8192 * plain / (2 * math.pi)
    assert np.allclose(f[turns > 4], plain[turns > 4]) and np.allclose(f[turns < 1], plain[turns < 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.all((f[mid] < plain[mid]) & (f[mid] > plain[mid] / 8))


@pytest.mark.parametrize("layout", ["halves", "pairs"])
def test_rope_quarter_turn(layout):
    # one pair at a quarter of a turn: (a, b) -> (-b, a); the tail stays
    x = np.array([[[1.0, 2.0, 7.0]]])
    y = oatt.rope(x, [1], np.array([math.pi / 2]), layout=layout)
    assert np.allclose(y, [[[-2.0, 1.0, 7.0]]], atol=1e-15)
    x = np.arange(1.0, 5.0).reshape(1, 1, 4)
    y = oatt.rope(x, [1], np.array([math.pi / 2, math.pi]), layout=layout)
    assert np.allclose(y, [[[-3.0, -2.0, 1.0, -4.0]]] if layout == "halves" else [[[-2.0, 1.0, -3.0, -4.0]]], atol=1e-14)


def test_rope_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 16))
    f = oatt.freqs(16)
    p = np.array([0, 3, 70, 4096, 100000])
    y = oatt.rope(x, p, f)
    assert np.allclose(np.linalg.norm(y, axis=2), np.linalg.norm(x, axis=2))
    assert np.allclose(oatt.rope(y, -p, f), x, atol=1e-9) and np.array_equal(y[0], x[0])
    # scores depend on the distance alone
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    a = np.sum(oatt.rope(q, [40], f) * oatt.rope(k, [33], f))
    b = np.sum(oatt.rope(q, [1007], f) * oatt.rope(k, [1000], f))
    assert np.isclose(a, b, rtol=1e-10)


# ------------------------------------------------------------------ the code formats

def test_e4m3_values():
    v = oatt.E4M3
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x7e] == 448.0
    assert np.isnan(v[0x7f]) and np.isnan(v[0xff]) and v[0xb8] == -1.0
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, v, equal_nan=True)


def test_encode_is_nearest_even():
    assert oatt.encode("i8", [0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 127.4, 300.0, -300.0]).view(np.int8).tolist() == \
        [0, 2, 2, 0, -2, 126, 127, 127, -127]
    y = np.array([0.0, 1.0, 1.0625, 1.1875, 17.0, 19.0, 448.0, 464.0, 1e9, 2.0 ** -10, 3 * 2.0 ** -10, -1.0625])
    assert oatt.E4M3[oatt.encode("e4m3", y)].tolist() == [0, 1, 1, 1.25, 16, 20, 448, 448, 448, 0, 2.0 ** -8, -1]
    rng = np.random.default_rng(1)
    y = rng.standard_normal(2000) * 10.0 ** rng.uniform(-4, 2, 2000)
    got = oatt.E4M3[oatt.encode("e4m3", y)]
    every = oatt.E4M3[np.isfinite(oatt.E4M3)]
    best = np.abs(every[None] - np.clip(y, -448, 448)[:, None]).min(1)
    assert np.array_equal(np.abs(got - np.clip(y, -448, 448)), best)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_least_scale(fmt):
    rng = np.random.default_rng(2)
    for a in np.concatenate((10.0 ** rng.uniform(-25, 30, 300), 127 * 2.0 ** rng.integers(-20, 20, 20), [448.0, 448.0001, 127.0])):
        a = float(np.float32(a))
        d = oatt.least_scale(fmt, a)
        top = oatt.LARGEST_CODE[fmt]
        step = d / 2 if fmt == "e4m3" else math.ldexp(1.0, math.frexp(d)[1] - 12)
        below = d - step if math.frexp(d)[0] != 0.5 or fmt == "e4m3" else d - step / 2
        assert top * d >= a > top * below
        assert np.float32(d) == d and (math.frexp(d)[0] * 4096) % 1 == 0
    assert oatt.least_scale(fmt, 0.0) == 2.0 ** -112 and oatt.least_scale(fmt, 3.4e38) == oatt.SCALE_MAX[fmt]
    assert oatt.least_scale("i8", 127.0) == 1.0 and oatt.least_scale("e4m3", 448.0) == 1.0
    assert oatt.least_scale("e4m3", 449.0) == 2.0


# ------------------------------------------------------------------ the cache

def empty(fmt, block, heads=1, dim=16, page=16, table=((0,),), n_pages=1):
    rng = np.random.default_rng(3)
    return au.cache_arrays(rng, fmt, n_pages, heads, page, dim, block, table)


def test_store_worked():
    c = empty("i8", 4)
    x = np.zeros((1, 1, 16))
    x[0, 0, :3] = [127.0, -1.0, 0.5]
    oatt.store(c, x, 2 * x, [0], [0])
    assert c["k_scale"][0, 0, 0] == 1.0 and c["v_scale"][0, 0, 0] == 2.0
    assert c["k"][0, 0, 0, :4].view(np.int8).tolist() == [127, -1, 0, 0]
    # a second token four times as large: the first one's codes are rounded again under its scale
    oatt.store(c, 4 * x, x, [0], [1])
    assert c["k_scale"][0, 0, 0] == 4.0 and c["v_scale"][0, 0, 0] == 2.0
    assert c["k"][0, 0, 0, :3].view(np.int8).tolist() == [32, 0, 0] and c["k"][0, 0, 1, :3].view(np.int8).tolist() == [127, -1, 0]
    assert c["v"][0, 0, 1, :3].view(np.int8).tolist() == [64, 0, 0]
    oatt.store(c, x, x, [0], [4])  # the next block
    assert c["k_scale"][0, 0, :2].tolist() == [4.0, 1.0]
    oatt.store(c, 0.5 * x, x, [0], [0])  # the block's first position starts it anew
    assert c["k_scale"][0, 0, 0] == 0.5


def test_store_not_finite():
    c = empty("e4m3", 2, heads=2)
    x = np.ones((1, 2, 16))
    x[0, 1, 5] = np.inf
    oatt.store(c, x, np.full((1, 2, 16), 3.0), [0], [2])
    assert c["k_scale"][0, 0, 1] == 2.0 ** -8 and np.isnan(c["k_scale"][0, 1, 1])
    k, v = oatt.load(c, [0], [2])
    assert np.array_equal(k[0, 0], np.ones(16)) and np.all(np.isnan(k[0, 1])) and np.array_equal(v[0], np.full((2, 16), 3.0))
    oatt.store(c, np.ones((1, 2, 16)), np.ones((1, 2, 16)), [0], [3])
    assert np.isnan(c["k_scale"][0, 1, 1])  # until its first position is written again
    oatt.store(c, np.ones((1, 2, 16)), np.ones((1, 2, 16)), [0], [2])
    assert c["k_scale"][0, 1, 1] == 2.0 ** -8


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("block", [1, 4, 16])
def test_store_error(fmt, block):
    # stored in one call: half a step of the largest value's scale (i8), of the value (e4m3)
    rng = np.random.default_rng(4)
    table, pages = au.shuffled_table(rng, [40, 23], 16)
    c = au.cache_arrays(rng, fmt, pages, 2, 16, 32, block, table)
    seq, pos = np.repeat([0, 1], [40, 23]), np.concatenate((np.arange(40), np.arange(23)))
    x = rng.standard_normal((2, 63, 2, 32)).astype(np.float32).astype(np.float64)
    oatt.store(c, x[0], x[1], seq, pos)
    for got, want in zip(oatt.load(c, seq, pos), x):
        d = 8.0 / 127 if fmt == "i8" else 0.0
        assert np.all(np.abs(got - want) <= 0.51 * d + np.abs(want) * 2.0 ** -4 * (fmt == "e4m3") + 2.0 ** -16)


def test_load_without_place():
    c = empty("i8", 4, table=((0, 7, -1),), n_pages=2)
    k, _ = oatt.load(c, [0, 0, 0, 1, -1, 0], [0, 16, 32, 0, 0, -1])
    assert np.any(k[0] != 0) and not np.any(k[1:])


# ------------------------------------------------------------------ attention

def test_attend_worked():
    # two keys with scores ln 3 apart: weights 3/4, 1/4
    c = empty("i8", 1, table=((0,),))
    c["k"][:] = 0
    c["v"][:] = 0
    c["k_scale"][:] = c["v_scale"][:] = 1.0
    c["k"][0, 0, 0, 0], c["k"][0, 0, 1, 0] = 2, 1
    c["v"][0, 0, 0, 1], c["v"][0, 0, 1, 1] = 8, 4
    q = np.zeros((2, 1, 16))
    q[:, 0, 0] = math.log(3.0)
    out, lse, _, _ = oatt.attend(c, q, [0, 0], [1, 0], scale=1.0)
    assert np.isclose(out[0, 0, 1], 7.0) and np.isclose(lse[0, 0], math.log(9 + 3)) and out[1, 0, 1] == 8.0
    out, lse, _, _ = oatt.attend(c, q[:1], [0], [1], scale=1.0, window=1)
    assert np.isclose(out[0, 0, 1], 4.0) and np.isclose(lse[0, 0], math.log(3.0))


def test_attend_rows_without_keys():
    c = empty("i8", 4, table=((-1,),))
    out, lse, _, _ = oatt.attend(c, np.ones((4, 2, 16)), [0, -1, 5, 0], [3, 3, 3, -1])
    assert not out.any() and np.all(lse == -np.inf)


def test_attend_is_a_mean():
    rng = np.random.default_rng(5)
    table, pages = au.shuffled_table(rng, [50], 16)
    c = au.cache_arrays(rng, "e4m3", pages, 2, 16, 32, 4, table)
    out, lse, _, _ = oatt.attend(c, np.zeros((1, 4, 32)), [0], [49])
    _, v = oatt.load(c, np.zeros(50, dtype=int), np.arange(50))
    assert np.allclose(out[0, 0], v[:, 0].mean(0)) and np.allclose(out[0, 3], v[:, 1].mean(0)) and np.allclose(lse, math.log(50))


def test_lost_low_parts_are_seen():
    rng = np.random.default_rng(6)
    table, pages = au.shuffled_table(rng, [400], 16)
    c = au.cache_arrays(rng, "i8", pages, 1, 16, 128, 16, table)
    q = rng.standard_normal((2, 8, 128))
    want, lse, mass, spread = oatt.attend(c, q, [0, 0], [399, 399])
    for n, seen in ((1, True), (2, False)):
        got = oatt.attend(c, au.exact_parts(q, n), [0, 0], [399, 399])[0]
        assert (au.norm_error(got, want) > au.NORM_TOL) == seen
        b, _ = au.attend_bounds(c, want, lse, mass, spread, 400, False)
        assert seen or np.all(np.abs(got - want) <= b)
