"""gf_attend on the GPU against the fp64 oracle: element by element and norm-wise."""

import numpy as np
import pytest

import attend_util as au
from gpu_util import assert_within, dev_tensor
from oracle import attend as oatt

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(scope="module")
def G(lib):
    yield lib
    assert lib.device_status() == 0


def call(G, dc, q, seq, pos, window=0, run=1, scale=0.0, ldq=0, ld_dst=0, at=0, lse=True, how="direct", seq_null=False,
         pad_ws=0):
    T, Hq, D = q.shape
    f16 = q.dtype == np.float16
    dt = torch.float16 if f16 else torch.float32
    H = dc.t["k"].shape[1]
    w, wd = ldq or Hq * D, ld_dst or Hq * D
    qt = torch.full((at + T * w + 8,), np.nan, dtype=dt, device="cuda")
    qt[at:at + T * w].view(T, w)[:, :Hq * D] = dev_tensor(q.reshape(T, -1))
    out = torch.full((at + T * wd + 8,), -77.0, dtype=dt, device="cuda")
    ls = torch.full((T * Hq + 4,), -77.0, device="cuda")
    ws = torch.full((G.attend_workspace(T, Hq, H, D, run) + pad_ws,), 0xff, dtype=torch.uint8, device="cuda")
    s = None if seq_null else dev_tensor(np.asarray(seq, dtype=np.int32))
    p = dev_tensor(np.asarray(pos, dtype=np.int32))
    args = (dc.cache, qt[at:], T, Hq, s, p, out[at:], ws)
    kw = dict(type=G.F16 if f16 else G.F32, ldq=ldq, ld_dst=ld_dst, scale=scale, window=window, run=run, lse=ls if lse else None)
    torch.cuda.synchronize()
    if how == "graph":
        g = G.Graph([G.prepare_attend(*args, **kw)])
        side = torch.cuda.Stream()
        g.launch(stream=side)
        g.launch(stream=side)
    else:
        G.attend(*args, **kw)
    torch.cuda.synchronize()
    rows = out[at:at + T * wd].view(T, wd)
    assert torch.all(rows[:, Hq * D:] == -77.0) and torch.all(out[:at] == -77.0) and torch.all(out[at + T * wd:] == -77.0)
    assert torch.all(ls[T * Hq if lse else 0:] == -77.0)
    return rows[:, :Hq * D].reshape(T, Hq, D).double().cpu().numpy(), ls[:T * Hq].view(T, Hq).double().cpu().numpy()


def check(G, c, q, seq, pos, window=0, scale=None, dc=None, norm=True, **kw):
    dc = dc or au.DeviceCache(G, c)
    want, lse, mass, spread = oatt.attend(c, q, seq, pos, scale, window)
    keys = np.array([[len(oatt.seen(c, int(s), int(p), window))] * q.shape[1] for s, p in zip(seq, pos)], dtype=np.float64)
    got, gl = call(G, dc, q, seq, pos, window=window, scale=scale or 0.0, **kw)
    f16 = q.dtype == np.float16
    b, bl = au.attend_bounds(c, want, lse, mass, spread, keys, f16)
    assert_within(got, want, b, "out")
    if kw.get("lse", True):
        empty = keys == 0
        assert np.array_equal(np.isneginf(gl), empty)
        assert_within(np.where(empty, 0, gl), np.where(empty, 0, lse), bl, "lse")
    assert not got[keys == 0].any()
    if norm and not f16 and want.any():
        assert au.norm_error(got, want) <= au.NORM_TOL
    return got, gl


def setup(rng, fmt, lengths, H, page, D, block, **kw):
    table, pages = au.shuffled_table(rng, lengths, page)
    return au.cache_arrays(rng, fmt, pages, H, page, D, block, table, **kw)


def queries(rng, T, Hq, D, f16=False, size=1.0):
    return (rng.standard_normal((T, Hq, D)) * size).astype(np.float16 if f16 else np.float32)


# H, group, D, page, block
HEADS = [(1, 1, 16, 16, 1), (2, 4, 64, 16, 16), (2, 4, 128, 64, 16), (1, 8, 128, 16, 4), (3, 5, 80, 32, 32), (2, 1, 96, 128, 64),
         (1, 16, 128, 64, 16), (2, 9, 64, 16, 8), (1, 2, 256, 64, 64), (2, 12, 256, 16, 2), (1, 7, 112, 16, 16), (1, 33, 48, 64, 1),
         (2, 3, 192, 32, 16)]
LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 200, 257, 500]


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("H, group, D, page, block", HEADS)
def test_lengths(G, H, group, D, page, block, fmt):
    rng = np.random.default_rng(D + group)
    c = setup(rng, fmt, LENGTHS, H, page, D, block)
    seq, pos = au.positions(LENGTHS, 1)
    dc = au.DeviceCache(G, c)
    check(G, c, queries(rng, len(seq), H * group, D), seq, pos, dc=dc)
    check(G, c, queries(rng, len(seq), H * group, D, True), seq, pos, dc=dc, seq_null=True)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("n", [1, 33, 1000, 3001])
@pytest.mark.parametrize("H, group, D", [(1, 1, 64), (8, 4, 128), (1, 8, 128), (1, 16, 128), (2, 8, 256)])
def test_one_sequence(G, H, group, D, n, fmt):
    """Few rows: an item's keys are spread over CTAs and joined."""
    rng = np.random.default_rng(n)
    c = setup(rng, fmt, [n], H, 64, D, 16)
    check(G, c, queries(rng, 1, H * group, D, size=2.0), [0], [n - 1], how="graph")


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("H, group, D", [(2, 4, 128), (1, 1, 64), (1, 8, 128), (2, 2, 256), (1, 5, 80), (1, 20, 64)])
@pytest.mark.parametrize("per, run", [(2, 2), (5, 5), (8, 8), (5, 1), (3, 4), (40, 40), (4, 64)])
def test_several_tokens(G, H, group, D, per, run, fmt):
    rng = np.random.default_rng(per + D)
    lengths = [40, 41, 100, 333, 64]
    c = setup(rng, fmt, lengths, H, 16, D, 4)
    seq, pos = au.positions(lengths, per)
    check(G, c, queries(rng, len(seq), H * group, D), seq, pos, run=run)


@pytest.mark.parametrize("run", [1, 3, 8, 64])
@pytest.mark.parametrize("window", [0, 1, 5, 16, 100])
def test_ragged_and_padded(G, run, window):
    """Runs of unequal length, tokens of no sequence between and behind them, windows, equal tokens."""
    rng = np.random.default_rng(window)
    lengths = [70, 300, 20, 129]
    c = setup(rng, "i8", lengths, 2, 32, 64, 8)
    seq = np.array([0] * 7 + [1] * 3 + [-1] + [2] * 20 + [3] + [9] + [3] * 4 + [1, 1] + [-1, -1], dtype=np.int32)
    pos = np.concatenate((np.arange(63, 70), [299, 5, 5], [3], np.arange(20), [128], [0], [128, 127, 0, 126], [-1, 298], [0, -1]))
    check(G, c, queries(rng, len(seq), 8, 64), seq, pos.astype(np.int32), window=window, run=run)


@pytest.mark.parametrize("window", [1, 17, 64, 1000])
@pytest.mark.parametrize("D, per", [(128, 1), (256, 3)])
def test_window(G, D, per, window):
    rng = np.random.default_rng(window)
    lengths = [3, 64, 65, 500, 1025]
    c = setup(rng, "e4m3", lengths, 1, 16, D, 16)
    # scales that lie before the window count for nothing
    for i, n in enumerate(lengths):
        for j in range(0, max(0, n - per - window - 16), 16):
            c["k_scale"][c["table"][i, j // 16], :, 0] = np.nan
            c["v_scale"][c["table"][i, j // 16], :, 0] = np.nan
    seq, pos = au.positions(lengths, per)
    check(G, c, queries(rng, len(seq), 4, D), seq, pos, window=window, run=per)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_behind_the_last_key(G, D):
    """What lies behind a sequence's last token in its page, and in pages of no sequence, is never seen."""
    rng = np.random.default_rng(D)
    lengths = [5, 18, 100]
    c = setup(rng, "i8", lengths, 2, 64, D, 1)
    for s, n in enumerate(lengths):
        for j in range(n, c["table"].shape[1] * 64):
            at = oatt.place(c, s, j)
            if at is not None:
                c["k_scale"][at[0], :, at[1]] = np.nan
                c["v_scale"][at[0], :, at[1]] = np.inf
                c["v"][at[0], :, at[1]] = 0x80
    spare = set(range(c["k"].shape[0])) - set(c["table"].ravel().tolist())
    c["k_scale"][list(spare)] = np.nan
    seq, pos = au.positions(lengths, 1)
    check(G, c, queries(rng, 3, 6, D), seq, pos)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_bad_pages(G, fmt):
    """Pages that the table does not have are not followed, their positions not seen."""
    rng = np.random.default_rng(1)
    c = setup(rng, fmt, [100, 100, 100, 100], 2, 16, 64, 16)
    t = c["table"]
    t[0, 2], t[0, 6] = -1, 1 << 30
    t[1, 0] = -2 ** 31
    t[2, :] = 2 ** 31 - 1
    t[3, 0], t[3, 1] = t[3, 1], t[3, 1]  # the same page twice
    seq = np.array([0, 1, 2, 3, 0, 1], dtype=np.int32)
    pos = np.array([99, 99, 99, 99, 40, 2 ** 31 - 1], dtype=np.int32)  # the last: beyond the table
    check(G, c, queries(rng, 6, 4, 64), seq, pos)
    check(G, c, queries(rng, 6, 4, 64), seq, pos, window=30)


def test_nan_block_is_seen(G):
    """A block that was stored with a value that is not finite makes the rows that see it NaN, no others."""
    rng = np.random.default_rng(2)
    c = setup(rng, "i8", [100, 100], 2, 16, 64, 16)
    c["k_scale"][c["table"][0, 3], 1, 0] = np.nan
    c["v_scale"][c["table"][1, 2], 0, 0] = np.nan
    seq, pos = np.array([0, 0, 1, 1], dtype=np.int32), np.array([99, 47, 99, 31], dtype=np.int32)
    q = queries(rng, 4, 4, 64)
    got, lse = call(G, au.DeviceCache(G, c), q, seq, pos)
    want = oatt.attend(c, q, seq, pos)[0]
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.isnan(got[0, 2:]).all() and np.isnan(got[2, :2]).all() and np.isfinite(got[1]).all() and np.isfinite(got[3]).all()
    assert np.isnan(lse[0, 2:]).all() and np.isfinite(lse[2]).all()


@pytest.mark.parametrize("D, window", [(64, 0), (128, 0), (256, 0), (128, 20)])
def test_nan_block_beside(G, D, window):
    """Rows that share their keys' reading with rows that see such a block, and do not see it themselves, are as
    without it."""
    rng = np.random.default_rng(12)
    c = setup(rng, "i8", [200], 1, 16, D, 16)
    seq, pos = np.zeros(4, dtype=np.int32), np.array([40, 100, 120, 199], dtype=np.int32)
    q = queries(rng, 4, 2, D)
    for name in ("k_scale", "v_scale"):
        bad = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in c.items()}
        bad[name][c["table"][0, 7], 0, 0] = np.nan  # positions 112 to 127: the token at 100 is of their chunk
        got, _ = call(G, au.DeviceCache(G, bad), q, seq, pos, run=4, window=window)
        want, lse, mass, spread = oatt.attend(c, q, seq, pos, window=window)
        sees = [p >= 112 and (not window or p - window < 127) for p in pos]
        b, _ = au.attend_bounds(c, want, lse, mass, spread, np.repeat(pos[:, None] + 1.0, 2, 1), False)
        for t in range(4):
            if sees[t]:
                assert np.isnan(got[t]).all()
            else:
                assert_within(got[t], want[t], b[t], "token %d" % t)


def test_captured_by_a_user(G):
    """Direct calls recorded by a capture of the user's own, replayed over changed inputs."""
    rng = np.random.default_rng(13)
    table, pages = au.shuffled_table(rng, [100, 100], 16)
    c = au.cache_arrays(rng, "i8", pages, 2, 16, 64, 4, table)
    dc = au.DeviceCache(G, c)
    k, v, q = (torch.empty(2, h, 64, device="cuda") for h in (2, 2, 8))
    out, turned = torch.empty_like(q), torch.empty_like(q)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    rot = torch.empty(G.rope_table_bytes(64), dtype=torch.uint8, device="cuda")
    G.rope_table(rot, 64)
    ws = torch.empty(G.attend_workspace(2, 8, 2, 64), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        G.rope(q, 2, 8, 64, pos, rot, turned)
        G.cache_store(dc.cache, k, v, 2, None, pos)
        G.attend(dc.cache, turned, 2, 8, None, pos, out, ws)
    for p in ([0, 7], [1, 8], [2, 9], [50, 99]):
        kn, vn, qn = (rng.standard_normal((2, h, 64)).astype(np.float32) for h in (2, 2, 8))
        for t, x in ((k, kn), (v, vn), (q, qn)):
            t.copy_(dev_tensor(x))
        pos.copy_(torch.tensor(p, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        oatt.store(c, kn, vn, [0, 1], p)
        want, lse, mass, spread = oatt.attend(c, turned.cpu().numpy(), [0, 1], p)
        b, _ = au.attend_bounds(c, want, lse, mass, spread, np.repeat(np.array(p, dtype=float)[:, None] + 1, 8, 1), False)
        assert_within(out.double().cpu().numpy(), want, b)
        assert np.array_equal(dc.host("k"), c["k"]) and np.array_equal(dc.host("v_scale"), c["v_scale"])


def test_hard_queries(G):
    """Zero, tiny, huge and not finite queries; scores far apart; a scale of its own."""
    rng = np.random.default_rng(3)
    c = setup(rng, "i8", [300], 1, 16, 128, 4)
    q = queries(rng, 8, 4, 128)
    q[0] = 0.0
    q[1] *= 1e-30
    q[2] *= 1e30
    q[3, 0, 5], q[3, 1, 7] = np.nan, np.inf
    q[4, :, 0] = 1e4   # one outlier
    q[5] *= 30.0
    q[6, 2] = np.float32(1e-42)
    seq, pos = np.zeros(8, dtype=np.int32), np.arange(292, 300, dtype=np.int32)
    got, lse = call(G, au.DeviceCache(G, c), q, seq, pos, run=8)
    assert np.isnan(got[3, :2]).all() and np.isnan(lse[3, :2]).all()
    fine = np.ones((8, 4), dtype=bool)
    fine[3, :2] = fine[2] = False
    q2 = np.where(np.isfinite(q), q, 0)
    want, wl, mass, spread = oatt.attend(c, q2, seq, pos)
    keys = np.repeat((pos + 1.0)[:, None], 4, 1)
    b, bl = au.attend_bounds(c, want, wl, mass, spread, keys, False)
    assert_within(got[fine], want[fine], b[fine], "out")
    assert_within(lse[fine], wl[fine], bl[fine], "lse")
    # scores 1e30 apart: the largest alone
    assert_within(got[2], want[2], 1e-5 * mass[2] + 1e-30, "huge")
    check(G, c, queries(rng, 3, 4, 128), [0, 0, 0], [10, 200, 299], scale=0.3)


@pytest.mark.parametrize("size", [1e-30, 1.0, 1e25])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_scales_of_values(G, fmt, size):
    """Values' scales that rise and fall by powers of ten along the sequence."""
    rng = np.random.default_rng(4)
    c = setup(rng, fmt, [700], 2, 16, 128, 16)
    e = rng.integers(-40, 1, c["v_scale"].shape)
    c["v_scale"] = (c["v_scale"] * 2.0 ** np.round(np.log2(size)) * 2.0 ** e).astype(np.float32)
    c["k_scale"] = (c["k_scale"] * 2.0 ** rng.integers(-6, 2, e.shape)).astype(np.float32)
    check(G, c, queries(rng, 2, 8, 128), [0, 0], [699, 350])


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("ldq, ld_dst, at", [(0, 0, 0), (600, 520, 0), (513, 515, 1), (640, 516, 2)])
def test_strides_and_alignment(G, ldq, ld_dst, at, f16):
    rng = np.random.default_rng(ldq)
    lengths = [40, 300, 7]
    c = setup(rng, "i8", lengths, 2, 16, 64, 16)
    seq, pos = au.positions(lengths, 1)
    check(G, c, queries(rng, 3, 8, 64, f16), seq, pos, ldq=ldq, ld_dst=ld_dst, at=at, lse=at != 1)


def test_many_short_rows(G):
    """More items than CTAs, most of a chunk or two."""
    rng = np.random.default_rng(5)
    lengths = list(rng.integers(1, 70, 300))
    c = setup(rng, "i8", lengths, 4, 16, 64, 4)
    seq, pos = au.positions(lengths, 1)
    check(G, c, queries(rng, 300, 8, 64), seq, pos)
    order = rng.permutation(300)
    check(G, c, queries(rng, 300, 8, 64), seq[order], pos[order])


def test_one_long_among_short(G):
    rng = np.random.default_rng(6)
    lengths = [9] * 20 + [5000] + [31] * 20
    c = setup(rng, "e4m3", lengths, 2, 64, 64, 16)
    seq, pos = au.positions(lengths, 1)
    check(G, c, queries(rng, 41, 8, 64), seq, pos, how="graph")


def test_a_prompt(G):
    """Every token of a prompt sees what is before it."""
    rng = np.random.default_rng(7)
    c = setup(rng, "i8", [260], 1, 16, 64, 16)
    check(G, c, queries(rng, 260, 4, 64), np.zeros(260, dtype=np.int32), np.arange(260, dtype=np.int32), run=260)


def test_repeatable_and_shared_workspace(G):
    """Equal bits on every run; two prepared calls that share a workspace, one after the other; two at once with
    workspaces of their own."""
    rng = np.random.default_rng(8)
    lengths = [1000, 33, 700]
    c = setup(rng, "i8", lengths, 2, 16, 128, 16)
    dc = au.DeviceCache(G, c)
    q = dev_tensor(queries(rng, 3, 8, 128))
    p, p2 = dev_tensor(np.array(lengths, dtype=np.int32) - 1), dev_tensor(np.array([10, 32, 699], dtype=np.int32))
    n = G.attend_workspace(3, 8, 2, 128)
    ws, other = (torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    want = [torch.empty(3, 8, 128, device="cuda") for _ in range(2)]
    for w, at in zip(want, (p, p2)):
        G.attend(dc.cache, q, 3, 8, None, at, w, ws)
    torch.cuda.synchronize()
    out = [torch.zeros(3, 8, 128, device="cuda") for _ in range(2)]
    one = G.Graph([G.prepare_attend(dc.cache, q, 3, 8, None, p, out[0], ws)])
    two = G.Graph([G.prepare_attend(dc.cache, q, 3, 8, None, p2, out[1], ws, pdl=True)])
    three = G.Graph([G.prepare_attend(dc.cache, q, 3, 8, None, p2, out[1], other)])
    side = torch.cuda.Stream()
    for rounds in range(20):
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        one.launch(stream=side)
        two.launch(stream=side)
        side.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        out[1].zero_()
        torch.cuda.synchronize()
        one.launch(stream=side)
        three.launch()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_positions_change_between_launches(G):
    rng = np.random.default_rng(9)
    c = setup(rng, "e4m3", [400, 400], 2, 32, 64, 8)
    dc = au.DeviceCache(G, c)
    q = queries(rng, 2, 4, 64)
    p, out = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, 4, 64, device="cuda")
    ws = torch.empty(G.attend_workspace(2, 4, 2, 64), dtype=torch.uint8, device="cuda")
    g = G.Graph([G.prepare_attend(dc.cache, dev_tensor(q), 2, 4, None, p, out, ws)])
    for pos in ([0, 399], [399, 0], [-1, 57], [200, 201], [-1, -1]):
        p.copy_(torch.tensor(pos, dtype=torch.int32))
        g.launch()
        torch.cuda.synchronize()
        want, lse, mass, spread = oatt.attend(c, q, [0, 1], pos)
        b, _ = au.attend_bounds(c, want, lse, mass, spread, np.repeat(np.array(pos, dtype=float)[:, None] + 1, 4, 1), False)
        assert_within(out.double().cpu().numpy(), want, b)


def test_far_into_a_large_pool(G):
    """Code offsets beyond 32 bits: the last pages of a large pool against the same pages of a small one."""
    H, page, D, block = 8, 64, 128, 16
    n_pages = (5 << 30) // (H * page * D)
    rng = np.random.default_rng(10)
    c = au.cache_arrays(rng, "i8", 4, H, page, D, block, [[2, 0, 3, 1]])
    dc = au.DeviceCache(G, c)
    q, pos = queries(rng, 1, 32, D), [250]
    want, wl = call(G, dc, q, [0], pos)
    k, v = (torch.zeros(n_pages, H, page, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((n_pages, H, page // block), float("nan"), device="cuda") for _ in range(2))
    for big, name in ((k, "k"), (v, "v"), (ks, "k_scale"), (vs, "v_scale")):
        big[-4:] = dc.t[name]
    table = dc.t["table"] + (n_pages - 4)
    far = au.DeviceCache.__new__(au.DeviceCache)
    far.t = dict(k=k, v=v, k_scale=ks, v_scale=vs, table=table)
    far.cache = G.Cache(k, v, ks, vs, G.CACHE_I8, n_pages, H, page, D, block, table, 1, 4)
    got, gl = call(G, far, q, [0], pos)
    assert np.array_equal(got, want) and np.array_equal(gl, wl)
