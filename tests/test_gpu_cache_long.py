"""gf_cache_store, gf_cache_load and gf_attend on the GPU in the forms that long calls take: four tokens a CTA in the
load, windows of 2 to 32 tokens with several blocks each in the store, batches beyond 256 rows, and calls of more
than 1024 rows to gf_attend.  Codes, scales and what is read back are compared bit for bit."""

import numpy as np
import pytest

import attend_util as au
from gpu_util import assert_within, dev_tensor
from oracle import attend as oatt
from test_gpu_attend import call, check, queries, setup
from test_gpu_cache import fmt_type, rows_on, same_cache, values

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(scope="module")
def G(lib):
    yield lib
    assert lib.device_status() == 0


def tokens_of(spans):
    """seq, pos of positions [a, b) of each sequence."""
    seq = np.concatenate([np.full(b - a, i) for i, (a, b) in enumerate(spans)]).astype(np.int32)
    return seq, np.concatenate([np.arange(a, b) for a, b in spans]).astype(np.int32)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("T", [1023, 1024, 1025, 1026, 1027, 4097])
@pytest.mark.parametrize("heads, dim, ld, at", [(2, 128, 0, 0), (3, 80, 0, 0), (1, 16, 0, 0), (2, 64, 136, 8), (2, 64, 131, 1)])
def test_long_loads(G, heads, dim, ld, at, T, fmt, f16):
    rng = np.random.default_rng(T + dim)
    table, pages = au.shuffled_table(rng, [700, 300], 16)
    c = au.cache_arrays(rng, fmt, pages, heads, 16, dim, 4, table)
    seq = rng.integers(-1, 3, T).astype(np.int32)  # -1 and 2: no such sequence
    pos = rng.integers(-5, 720, T).astype(np.int32)
    pos[T // 2:T // 2 + 9] = -1
    seq[-2:] = -1
    want = oatt.load(c, seq, pos)
    dc = au.DeviceCache(G, c)
    dt, w = torch.float16 if f16 else torch.float32, ld or heads * dim
    out = [torch.full((at + T * w + 8,), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    G.cache_load(dc.cache, T, dev_tensor(seq), dev_tensor(pos), out[0][at:], out[1][at:], type=G.F16 if f16 else G.F32, ldk=ld, ldv=ld)
    for o, x in zip(out, want):
        rows = o[at:at + T * w].view(T, w)
        assert torch.equal(rows[:, :heads * dim].cpu(), torch.from_numpy(x.reshape(T, -1).astype(np.float32)).to(dt))
        assert torch.all(rows[:, heads * dim:] == 7.0) and torch.all(o[:at] == 7.0) and torch.all(o[at + T * w:] == 7.0)


# heads, dim, page, block: with 8191 tokens the windows of both the plan of whole CTAs and that of a warp's blocks
LONG = [(8, 128, 64, 32), (8, 128, 64, 64), (8, 128, 16, 16), (2, 256, 128, 64), (4, 64, 32, 8), (5, 80, 64, 64)]


def ragged(rng, T, n):
    """n lengths that add up to T, each at least one."""
    cuts = np.sort(rng.choice(np.arange(1, T), n - 1, replace=False))
    return np.diff(np.concatenate(([0], cuts, [T])))


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("T, n", [(300, 40), (1500, 9), (8191, 7), (4001, 250)])
@pytest.mark.parametrize("heads, dim, page, block", LONG)
def test_long_stores(G, heads, dim, page, block, T, n, fmt):
    """Prompts behind tokens that were there, many blocks to a window."""
    rng = np.random.default_rng(T + n + block)
    before, news = rng.integers(0, 2 * block, n), ragged(rng, T, n)
    table, pages = au.shuffled_table(rng, before + news, page)
    c = au.cache_arrays(rng, fmt, pages, heads, page, dim, block, table)
    dc = au.DeviceCache(G, c)
    seq, pos = tokens_of(list(zip(before, before + news)))
    k, v = values(rng, (T, heads, dim), False), values(rng, (T, heads, dim), False)
    G.cache_store(dc.cache, dev_tensor(k), dev_tensor(v), T, dev_tensor(seq), dev_tensor(pos))
    oatt.store(c, k, v, seq, pos)
    same_cache(dc, c)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("T, n", [(300, 40), (8191, 7), (4001, 250)])
@pytest.mark.parametrize("heads, dim, page, block", LONG)
def test_long_stores_with_rotation(G, heads, dim, page, block, T, n, layout):
    """Equal, bit for bit, to gf_rope followed by the store of its results: a window's blocks take turns in one place
    for their cosines."""
    rng = np.random.default_rng(T + n + dim)
    Hq, n_rot = 2 * heads, dim // 16 * 8
    before, news = rng.integers(0, 2 * block, n), ragged(rng, T, n)
    table, pages = au.shuffled_table(rng, before + news, page)
    table[n // 2, 0] = -1  # some tokens have no place
    c = au.cache_arrays(rng, "i8", pages, heads, page, dim, block, table)
    a, b = au.DeviceCache(G, c), au.DeviceCache(G, c)
    seq, pos = (dev_tensor(x) for x in tokens_of(list(zip(before, before + news))))
    k, v, q = (dev_tensor(values(rng, (T, h, dim), False)) for h in (heads, heads, Hq))
    rot = torch.empty(G.rope_table_bytes(n_rot), dtype=torch.uint8, device="cuda")
    G.rope_table(rot, n_rot, base=500000.0)
    kr, qr, got = torch.empty_like(k), torch.empty_like(q), torch.full_like(q, 7.0)
    G.rope(k, T, heads, dim, pos, rot, kr, n_rot=n_rot, layout=layout)
    G.rope(q, T, Hq, dim, pos, rot, qr, n_rot=n_rot, layout=layout)
    placed = dev_tensor(np.array([oatt.place(c, s, p) is not None for s, p in zip(seq.tolist(), pos.tolist())]))
    qr[~placed] = 7.0
    G.cache_store(b.cache, kr, v, T, seq, pos)
    G.cache_store(a.cache, k, v, T, seq, pos, rope=rot, n_rot=n_rot, layout=layout, q=q, q_heads=Hq, q_dst=got)
    assert torch.equal(got, qr)
    for name in ("k_scale", "v_scale", "k", "v"):
        assert torch.equal(a.t[name], b.t[name]), name


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("block", [1, 4, 16, 64])
@pytest.mark.parametrize("T", [256, 257, 300, 1100])
def test_wide_decode_batches(G, T, block, f16):
    """One token of each of many sequences, in and at the start of blocks."""
    rng = np.random.default_rng(T + block)
    heads, dim, page = 2, 64, 64
    pos = rng.integers(0, 2 * block, T).astype(np.int32)
    table, pages = au.shuffled_table(rng, pos + 1, page)
    c = au.cache_arrays(rng, "i8", pages, heads, page, dim, block, table)
    dc = au.DeviceCache(G, c)
    k, v = values(rng, (T, heads, dim), f16), values(rng, (T, heads, dim), f16)
    G.cache_store(dc.cache, rows_on(k), rows_on(v), T, None, dev_tensor(pos), type=fmt_type(G, k))
    oatt.store(c, k, v, np.arange(T), pos)
    same_cache(dc, c)


@pytest.mark.parametrize("T, per, run", [(1023, 1, 1), (1025, 1, 1), (1100, 1, 1), (2100, 1, 1), (1100, 5, 5), (2100, 3, 4), (1100, 1, 7)])
def test_many_rows(G, T, per, run):
    """More than 32 groups of 32 rows, most of a chunk or two; some of no sequence."""
    rng = np.random.default_rng(T + per)
    lengths = list(rng.integers(per, 50, T // per))
    c = setup(rng, "i8", lengths, 2, 16, 64, 4)
    seq, pos = au.positions(lengths, per)
    seq = seq.copy()
    seq[rng.integers(0, len(seq), 40)] = -1
    check(G, c, queries(rng, len(seq), 4, 64), seq, pos, run=run)


@pytest.mark.parametrize("T", [65536, 65535])
def test_most_rows(G, T):
    """As many rows as a call may have, each of a sequence of one token: its value, or nothing."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    H, D, page = 1, 64, 16
    k, v = (torch.randint(1, 120, (T, H, page, D), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.full((T, H, 1), 1.0 / 64, device="cuda") for _ in range(2))
    table = torch.randperm(T, generator=g, device="cuda").int().view(T, 1).contiguous()
    cache = G.Cache(k, v, ks, vs, G.CACHE_I8, T, H, page, D, 16, table, T, 1)
    q, out = torch.randn(T, H, D, generator=g, device="cuda"), torch.empty(T, H, D, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos[::1000] = -1
    ws = torch.empty(G.attend_workspace(T, H, H, D), dtype=torch.uint8, device="cuda")
    G.attend(cache, q, T, H, None, pos, out, ws)
    want = v[table[:, 0].long(), :, 0].float() / 64
    want[::1000] = 0
    # one weight of 1 and a code: exact but for the unit's products and a division, 2^-20 as in attend_bounds
    assert bool(torch.all((out - want).abs() <= want.abs() * 2.0 ** -20))
