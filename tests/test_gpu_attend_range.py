"""gf_attend on the GPU where the values' scales of a sequence lie far apart: a block of large values that a row
gives no weight, or does not see, takes nothing from the others."""

import numpy as np
import pytest

import attend_util as au
from gpu_util import assert_within
from oracle import attend as oatt
from test_gpu_attend import call, check, queries, setup

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(scope="module")
def G(lib):
    yield lib
    assert lib.device_status() == 0


LOWEST = {"i8": 0x81, "e4m3": 0xfe}  # the codes of -127 and -448


def no_zeros(codes):
    """A large value that is zero would leave its element to the small ones."""
    return np.where(codes & 0x7f, codes, codes | 0x18).astype(np.uint8)


def blocks_at(c, s, blocks):
    """(page, block of the page) of blocks of sequence s."""
    per = c["k"].shape[2] // c["block"]
    return [(int(c["table"][s, b // per]), b % per) for b in blocks]


def repel(c, s, blocks, q, weight=100.0):
    """Keys of these blocks, by their first element alone, score `weight` and more below what the others make of it."""
    D, H = c["k"].shape[3], c["k"].shape[1]
    c["k"][..., 0] = 0
    least = c["k_scale"].min() * {"i8": 127.0, "e4m3": 448.0}[c["fmt"]]
    q[..., 0] = np.float32((weight + 40.0) * np.sqrt(D) / least)  # (others' scores lie within some 20 of zero)
    for p, b in blocks_at(c, s, blocks):
        c["k"][p, :, b * c["block"]:(b + 1) * c["block"], 0] = LOWEST[c["fmt"]]


def one_sequence(c, q, seq, pos, window=0):
    """The oracle's attend for rows that are all of sequence 0, or of none (pos < 0), at once."""
    T, Hq, D = q.shape
    n, H = int(max(pos)) + 1, c["k"].shape[1]
    k, v = (x.transpose(1, 0, 2) for x in oatt.load(c, np.zeros(n, dtype=int), np.arange(n)))  # [H, n, D]
    x = q.astype(np.float64).reshape(T, H, Hq // H, D).transpose(1, 0, 2, 3).reshape(H, -1, D) * D ** -0.5
    p = np.repeat(np.asarray(pos), Hq // H)[:, None]
    sees = (np.arange(n) <= p) & ((np.arange(n) > p - window) if window else True)
    a = np.where(sees, x @ k.transpose(0, 2, 1), -np.inf)
    m = a.max(-1, keepdims=True)
    e = np.exp(a - np.where(np.isfinite(m), m, 0.0))
    z = e.sum(-1, keepdims=True)
    w = e / np.where(z > 0, z, 1.0)
    spread = np.where(sees, np.abs(x) @ np.abs(k).transpose(0, 2, 1), 0.0).max(-1)
    with np.errstate(divide="ignore"):
        lse = np.where(z > 0, m + np.log(z), -np.inf)[..., 0]

    def rows(y):
        return y.reshape((H, T, Hq // H) + y.shape[2:]).swapaxes(0, 1).reshape((T, Hq) + y.shape[2:])
    return rows(w @ v), rows(lse), rows(w @ np.abs(v)), rows(spread)


def test_one_sequence_is_the_oracle():
    rng = np.random.default_rng(0)
    c = setup(rng, "i8", [50], 2, 16, 16, 4)
    q, pos = queries(rng, 6, 6, 16), [3, -1, 49, 20, 0, 30]
    for window in (0, 7):
        for a, b in zip(one_sequence(c, q, [0] * 6, pos, window), oatt.attend(c, q, np.zeros(6, dtype=int), pos, window=window)):
            assert np.allclose(a, b, rtol=1e-12, atol=1e-14)


def bounds_beside(c, q, seq, pos, window, blocks, attend=oatt.attend):
    """attend_bounds with the scores of the keys that have weight, and all of what the blocks contribute: their keys'
    scores are large, and so are their errors, but they have no weight to be wrong."""
    want, lse, mass, spread = attend(c, q, seq, pos, window=window)
    rest = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in c.items()}
    for p, b in blocks:
        rest["v"][p, :, b * c["block"]:(b + 1) * c["block"]] = 0
        rest["k"][p, :, b * c["block"]:(b + 1) * c["block"]] = 0
    without = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in rest.items()}
    without["k"] = c["k"]
    _, _, mass_rest, _ = attend(without, q, seq, pos, window=window)
    spread = attend(rest, q, seq, pos, window=window)[3]
    keys = np.repeat(np.clip(np.asarray(pos, dtype=np.float64) + 1, 0, window or None)[:, None], q.shape[1], 1)
    b, bl = au.attend_bounds(c, want, lse, mass_rest, spread, keys, False)
    return want, lse, b + (mass - mass_rest), bl


def where_of(where, n, block):
    last = (n - 1) // block
    return {"first": [0], "middle": [last // 2], "last": [last], "half": list(range(last // 2 + 1))}[where]


# H, group, D, page, block
SHAPES = [(1, 4, 128, 64, 16), (2, 1, 64, 16, 4), (1, 16, 128, 16, 1), (1, 8, 256, 64, 32), (1, 4, 96, 32, 8), (1, 12, 64, 64, 64)]


@pytest.mark.parametrize("where", ["first", "middle", "last", "half"])
@pytest.mark.parametrize("ratio", [10, 20, 40, 90])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("H, group, D, page, block", SHAPES)
def test_large_values_without_weight(G, H, group, D, page, block, fmt, ratio, where):
    """Weights below e^-100, values 2^ratio times the others': they count for nothing."""
    rng = np.random.default_rng(D + ratio)
    n = 1000
    c = setup(rng, fmt, [n], H, page, D, block)
    q = queries(rng, 1, H * group, D)
    which = where_of(where, n, block)
    repel(c, 0, which, q)
    at = blocks_at(c, 0, which)
    for p, b in at:
        c["v_scale"][p, :, b] *= np.float32(2.0 ** ratio)
    seq, pos = [0], [n - 1]
    want, lse, b, bl = bounds_beside(c, q, seq, pos, 0, at)
    got, gl = call(G, au.DeviceCache(G, c), q, seq, pos)
    assert_within(got, want, b, "out")
    assert_within(gl, lse, bl, "lse")
    assert au.norm_error(got, want) <= au.NORM_TOL


@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("ratio", [20, 40, 100])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("group, D", [(2, 64), (2, 128), (4, 128), (2, 256), (1, 80)])
def test_large_values_beside(G, group, D, fmt, ratio, window):
    """Rows that share their keys' reading with rows that see a block of large values, and do not see it themselves, are
    right by their own measure, as are those that do."""
    rng = np.random.default_rng(ratio + D)
    c = setup(rng, fmt, [200], 1, 16, D, 16)
    c["v"][c["table"][0, 7]] = no_zeros(c["v"][c["table"][0, 7]])
    c["v_scale"][c["table"][0, 7]] *= np.float32(2.0 ** ratio)  # positions 112 to 127
    seq, pos = np.zeros(4, dtype=np.int32), np.array([40, 100, 120, 199], dtype=np.int32)
    dc = au.DeviceCache(G, c)
    q = queries(rng, 4, group, D)
    got, _ = check(G, c, q, seq, pos, window=window, dc=dc, run=4)
    want = oatt.attend(c, q, seq, pos, window=window)[0]
    for t in range(4):
        assert au.norm_error(got[t], want[t]) <= au.NORM_TOL, t


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_that_come_and_go(G, D, fmt):
    """Each block of 32 keys has more weight than all before it, and values of quite another size."""
    rng = np.random.default_rng(D)
    n, block = 640, 32
    c = setup(rng, fmt, [n], 1, 64, D, block)
    q = queries(rng, 1, 4, D, size=0.02)
    c["k"][..., 0] = 0
    q[..., 0] = np.float32(2.0 * np.sqrt(D))
    one = {"i8": lambda v: v & 0xff, "e4m3": lambda v: int(oatt.encode("e4m3", np.array([float(v)]))[0])}[fmt]
    for i in range(n // block):  # scores rise by 5 a block or so
        (p, b), = blocks_at(c, 0, [i])
        c["k"][p, :, b * block:(b + 1) * block, 0] = one(i * 5)
        c["k_scale"][p, :, b] = 0.5
        c["v_scale"][p, :, b] = np.float32(2.0 ** [-60, 3, -20, 40, -7][i % 5])
    c["v"] = no_zeros(c["v"])
    for last in (n - 1, 400, 330, 100):
        check(G, c, q, [0], [last], norm=False)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("D, group", [(64, 1), (128, 4), (128, 16), (256, 2)])
@pytest.mark.parametrize("size", [1e20, 1e30, 1e34, 1e36])
def test_lowest_scores(G, size, D, group, fmt):
    """Scores far below zero, all of them: one key is seen whatever its score, and the largest of many is alone."""
    rng = np.random.default_rng(D)
    n, block = 1500, 4
    c = setup(rng, fmt, [n], 1, 16, D, block)
    one = {"i8": lambda v: v, "e4m3": lambda v: int(oatt.encode("e4m3", np.array([float(v)]))[0])}[fmt]
    c["k"][:] = one(96)
    c["k_scale"][:] = 1.0 / 64
    best = 1000  # the key whose score is the largest, and the last one's the next
    p, s = oatt.place(c, 0, best)
    c["k"][p, :, s] = one(32)
    p, s = oatt.place(c, 0, n - 1)
    c["k"][p, :, s] = one(64)
    dc = au.DeviceCache(G, c)
    for last, window in ((0, 0), (n - 1, 1), (n - 1, 0), (n - 1, 400), (best, 0), (40, 0)):
        q = np.full((1, group, D), -size, dtype=np.float32)
        if last == 40:  # neighbours' scores: the middle one the largest
            p, s = oatt.place(c, 0, 20)
            c["k"][p, :, s] = one(48)
            dc = au.DeviceCache(G, c)
        want, lse, mass, _ = oatt.attend(c, q, [0], [last], window=window)
        assert np.isfinite(lse).all() and (lse < -1e18).all()
        got, gl = call(G, dc, q, [0], [last], window=window)
        # one weight of 1: its parts, the matrix unit, the joining and the division, as attend_bounds counts them
        rel = 2.0 ** -20 + (1500 / 16 + 300) * 4 * au.U
        assert_within(got, want, mass * rel + 1e-30, "out")
        # q exactly so in two parts to 2^-22, D / 16 instructions 2^-22 each, and ten roundings
        assert_within(gl, lse, np.abs(lse) * (2.0 ** -22 * (1 + D / 16) + 10 * au.U), "lse")


def test_lowest_scores_of_two_parts(G):
    """Sequences whose scores are all low are joined from many warps' parts, beside ones that see nothing."""
    rng = np.random.default_rng(20)
    c = setup(rng, "i8", [900, 900], 2, 16, 64, 16)
    c["k"][:] = 64
    c["k_scale"][:] = 1.0
    q = np.full((3, 4, 64), -1e33, dtype=np.float32)
    want, lse, mass, _ = oatt.attend(c, q, [0, -1, 1], [899, 0, 700])
    got, gl = call(G, au.DeviceCache(G, c), q, [0, -1, 1], [899, 0, 700])
    assert_within(got, want, mass * (2.0 ** -20 + 400 * 4 * au.U) + 1e-30, "out")
    assert not got[1].any() and np.isneginf(gl[1]).all()
    assert np.all(np.abs(gl[[0, 2]] - lse[[0, 2]]) <= np.abs(lse[[0, 2]]) * (2.0 ** -22 * 5 + 10 * au.U))


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("D, group, n", [(64, 1, 40), (64, 2, 3000), (128, 4, 3000), (128, 16, 700), (256, 2, 1000), (128, 4, 20000)])
def test_largest_values(G, D, group, n, fmt):
    """Values as large as the format holds: their mean is no larger, whatever the number of keys."""
    rng = np.random.default_rng(n)
    c = setup(rng, fmt, [n], 1, 64, D, 16)
    c["v"] = (rng.integers(0x68, 0x7f, c["v"].shape)).astype(np.uint8)  # i8: 104 to 126, e4m3: 64 to 416
    c["v"][..., 5] |= 0x80 if fmt == "e4m3" else 0
    c["v_scale"][:] = 2.0 ** {"i8": 121, "e4m3": 119}[fmt]
    check(G, c, queries(rng, 1, group, D, size=0.1), [0], [n - 1])
    c["v_scale"][:] = 2.0 ** -90  # (bounds reach down to 1e-30)
    check(G, c, queries(rng, 1, group, D, size=0.1), [0], [n - 1])


@pytest.mark.parametrize("where", ["middle", "half", "stripes"])
@pytest.mark.parametrize("ratio", [-40, 20, 90])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("group, D, rows, run", [(4, 128, 80, 1), (16, 128, 70, 1), (8, 64, 80, 1), (3, 256, 70, 1), (4, 128, 160, 4)])
def test_large_values_within_a_warp(G, group, D, rows, run, fmt, ratio, where):
    """As test_large_values_without_weight, with so many rows over one sequence that each warp takes many chunks of it
    in turn; blocks of two chunks."""
    rng = np.random.default_rng(D + ratio + rows)
    n, block, H = 1500, 64, 4
    c = setup(rng, fmt, [n], H, 64, D, block)
    q = queries(rng, rows, H * group, D)
    last = (n - 1) // block
    which = list(range(1, last, 3)) if where == "stripes" else where_of(where, n, block)
    repel(c, 0, which, q)
    at = blocks_at(c, 0, which)
    for p, b in at:
        c["v_scale"][p, :, b] *= np.float32(2.0 ** ratio)
    pos = np.full(rows, n - 1, dtype=np.int32) - rng.integers(0, 3, rows).astype(np.int32)
    pos[::7] = -1  # (and some rows see nothing)
    seq = np.zeros(rows, dtype=np.int32)
    want, lse, b, bl = bounds_beside(c, q, seq, pos, 0, at, one_sequence)
    got, gl = call(G, au.DeviceCache(G, c), q, seq, pos, run=run)
    assert_within(got, want, b, "out")
    seen = pos >= 0
    assert_within(gl[seen], lse[seen], bl[seen], "lse")
    assert np.isneginf(gl[~seen]).all()
    for t in np.flatnonzero(seen):
        assert au.norm_error(got[t], want[t]) <= au.NORM_TOL, t


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_that_come_and_go_within_a_warp(G, D, fmt):
    """As test_scales_that_come_and_go, and its scores falling too: the first blocks have all the weight."""
    rng = np.random.default_rng(D + 1)
    n, block, rows = 1280, 64, 90
    c = setup(rng, fmt, [n], 4, 64, D, block)
    q = queries(rng, rows, 16, D, size=0.02)
    c["k"][..., 0] = 0
    q[..., 0] = np.float32(2.0 * np.sqrt(D)) * rng.choice([-1.0, 1.0, 0.1, -0.1], (rows, 16)).astype(np.float32)
    one = {"i8": lambda v: v & 0xff, "e4m3": lambda v: int(oatt.encode("e4m3", np.array([float(v)]))[0])}[fmt]
    for i in range(n // block):
        (p, b), = blocks_at(c, 0, [i])
        c["k"][p, :, b * block:(b + 1) * block, 0] = one(i * 5)
        c["k_scale"][p, :, b] = 0.5
        c["v_scale"][p, :, b] = np.float32(2.0 ** [-60, 3, -20, 40, -7, -7, 70, -90][i % 8])
    c["v"] = no_zeros(c["v"])
    seq, pos = np.zeros(rows, dtype=np.int32), np.full(rows, n - 1, dtype=np.int32)
    want, lse, mass, spread = one_sequence(c, q, seq, pos)
    got, gl = call(G, au.DeviceCache(G, c), q, seq, pos)
    b, bl = au.attend_bounds(c, want, lse, mass, spread, np.full(lse.shape, float(n)), False)
    assert_within(got, want, b, "out")
    assert_within(gl, lse, bl, "lse")


def dropped(c, q, pos):
    """What keys with weights below 2^-125 contribute: they may count as zero."""
    T, Hq, D = q.shape
    n, H = int(max(pos)) + 1, c["k"].shape[1]
    k, v = (x.transpose(1, 0, 2) for x in oatt.load(c, np.zeros(n, dtype=int), np.arange(n)))
    a = q.astype(np.float64).reshape(T, H, -1, D).transpose(1, 0, 2, 3).reshape(H, -1, D) * D ** -0.5 @ k.transpose(0, 2, 1)
    a = np.where(np.arange(n) <= np.repeat(pos, Hq // H)[:, None], a, -np.inf)
    w = np.exp(a - a.max(-1, keepdims=True))
    w[w >= 2.0 ** -125] = 0.0
    return (w @ np.abs(v)).reshape(H, T, Hq // H, D).swapaxes(0, 1).reshape(q.shape)


# (values' exponent, scores' level in powers of two) of a sequence's blocks
BLOCKS = {
    # a unit that falls, a maximum that comes while it serves, and large values whose weights make them count
    "weights that just count": [(52, 0), (22, -15), (18, 58), (53, 24), (31, 20)],
    # ever larger values, none of weight, between two blocks that have all of it
    "steps up": [(-55, 62)] + [(-45 + 10 * i, -62) for i in range(11)] + [(-55, 60)],
    "steps up and down": [(-30, 40)] + [(-22 + 8 * i, -60) for i in range(12)] + [(70 - 8 * i, -50) for i in range(12)] + [(-30, 44)],
    "ever more weight": [(60, -100), (30, -60), (0, -20), (-30, 20), (-60, 60), (-90, 110)],
    "ever less weight": [(-90, 110), (-60, 60), (-30, 20), (0, -20), (30, -60), (60, -100)],
    "more weight within a unit": [(20, -100), (19, -40), (18, 0), (17, 30), (90, -35), (-20, 50), (-21, 90)],
}


@pytest.mark.parametrize("blocks", list(BLOCKS))
@pytest.mark.parametrize("block", [16, 32, 64])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("group, D", [(2, 128), (10, 64), (2, 256)])
def test_scores_and_scales_by_blocks(G, group, D, fmt, block, blocks):
    """Blocks of any weight with values of any size: so many rows of one sequence that a warp takes most of it in turn."""
    rng = np.random.default_rng(D + block)
    rows, H, n = 480, 4, len(BLOCKS[blocks]) * block
    c = setup(rng, fmt, [n], H, 64, D, block)
    c["v"] = no_zeros(c["v"])
    q = queries(rng, rows, H * group, D, size=0.02 if fmt == "i8" else 0.005)  # (within a block scores lie close)
    q[..., 0] = np.float32(np.sqrt(D) * np.log(2.0))
    one = {"i8": lambda v: v & 0xff, "e4m3": lambda v: int(oatt.encode("e4m3", np.array([float(v)]))[0])}[fmt]
    c["k_scale"][:] = 1.0
    for i, (e, level) in enumerate(BLOCKS[blocks]):
        (p, b), = blocks_at(c, 0, [i])
        c["k"][p, :, b * block:(b + 1) * block, 0] = one(level)
        c["v_scale"][p, :, b] *= np.float32(2.0 ** e)
    seq, pos = np.zeros(rows, dtype=np.int32), n - 1 - rng.integers(0, 5, rows).astype(np.int32)
    want, lse, mass, spread = one_sequence(c, q, seq, pos)
    got, gl = call(G, au.DeviceCache(G, c), q, seq, pos)
    b, bl = au.attend_bounds(c, want, lse, mass, spread, np.full(lse.shape, float(n)), False)
    assert_within(got, want, b + dropped(c, q, pos), "out")
    assert_within(gl, lse, bl, "lse")
