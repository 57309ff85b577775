"""gf_cache_store and gf_cache_load on the GPU: codes and scales equal the oracle's exactly."""

import numpy as np
import pytest

import attend_util as au
from gpu_util import dev_tensor
from oracle import attend as oatt

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(scope="module")
def G(lib):
    yield lib
    assert lib.device_status() == 0


def values(rng, shape, f16):
    x = rng.standard_normal(shape) * np.exp(rng.uniform(-2, 2, shape[:2] + (1,)))
    return x.astype(np.float16 if f16 else np.float32)


def rows_on(x, ld=0, at=0):
    """[T, H, D] as device rows ld elements apart, `at` elements into the buffer."""
    T, w = x.shape[0], int(np.prod(x.shape[1:]))
    t = torch.full((at + T * (ld or w) + 8,), 3.0, dtype=torch.float16 if x.dtype == np.float16 else torch.float32, device="cuda")
    t[at:at + T * (ld or w)].view(T, -1)[:, :w] = dev_tensor(x.reshape(T, w))
    return t[at:]


def same_cache(dc, c):
    for name in ("k_scale", "v_scale", "k", "v"):
        assert np.array_equal(dc.host(name), c[name], equal_nan=c[name].dtype != np.uint8), name


def fmt_type(G, x):
    return G.F16 if x.dtype == np.float16 else G.F32


# heads, dim, page, block
CACHES = [(1, 16, 16, 1), (2, 64, 16, 16), (8, 128, 64, 16), (3, 80, 32, 4), (2, 96, 64, 64), (5, 256, 128, 32), (1, 112, 16, 2),
          (4, 240, 1024, 8)]


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("heads, dim, page, block", CACHES)
def test_prompt_then_steps(G, heads, dim, page, block, fmt, f16):
    rng = np.random.default_rng(dim + block)
    lengths = [37, 1, 100, 64]
    steps = 5
    table, pages = au.shuffled_table(rng, [n + steps for n in lengths], page)
    c = au.cache_arrays(rng, fmt, pages, heads, page, dim, block, table)
    dc = au.DeviceCache(G, c)
    # prompts, ragged, in two parts that cut blocks
    for part in range(2):
        spans = [(0, n // 3) if part == 0 else (n // 3, n) for n in lengths]
        seq = np.concatenate([np.full(b - a, i) for i, (a, b) in enumerate(spans)]).astype(np.int32)
        pos = np.concatenate([np.arange(a, b) for a, b in spans]).astype(np.int32)
        k, v = values(rng, (len(seq), heads, dim), f16), values(rng, (len(seq), heads, dim), f16)
        G.cache_store(dc.cache, dev_tensor(k), dev_tensor(v), len(seq), dev_tensor(seq), dev_tensor(pos), type=fmt_type(G, k))
        oatt.store(c, k, v, seq, pos)
        same_cache(dc, c)
    # decode steps: token t of sequence t, one of them padding
    call = None
    k, v = (torch.empty(4, heads, dim, dtype=torch.float16 if f16 else torch.float32, device="cuda") for _ in range(2))
    p = torch.empty(4, dtype=torch.int32, device="cuda")
    call = G.Graph([G.prepare_cache_store(dc.cache, k, v, 4, None, p, type=G.F16 if f16 else G.F32)])
    for s in range(steps):
        pos = np.array(lengths, dtype=np.int32) + s
        pos[s % 4] = -1 if s == 3 else pos[s % 4]
        kn, vn = values(rng, (4, heads, dim), f16), values(rng, (4, heads, dim), f16)
        k.copy_(dev_tensor(kn))
        v.copy_(dev_tensor(vn))
        p.copy_(dev_tensor(pos))
        call.launch()
        oatt.store(c, kn, vn, np.arange(4), pos)
        same_cache(dc, c)
    seq = np.concatenate([np.full(n + steps, i) for i, n in enumerate(lengths)] + [[4, -1, 0, 0]]).astype(np.int32)
    pos = np.concatenate([np.arange(n + steps) for n in lengths] + [[0, 0, -1, 1 << 20]]).astype(np.int32)
    want = oatt.load(c, seq, pos)
    for typ, dt in ((G.F32, torch.float32), (G.F16, torch.float16)):
        out = [torch.full((len(seq), heads, dim), 9.0, dtype=dt, device="cuda") for _ in range(2)]
        G.cache_load(dc.cache, len(seq), dev_tensor(seq), dev_tensor(pos), *out, type=typ)
        for o, w in zip(out, want):
            assert torch.equal(o.cpu(), torch.from_numpy(w.astype(np.float32)).to(dt))  # code * scale is exact in 32 bits


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("T", [300, 1000])
@pytest.mark.parametrize("heads, dim, page, block", [(2, 128, 64, 64), (1, 256, 64, 64), (3, 64, 64, 32), (2, 80, 16, 16)])
def test_long_prompts(G, heads, dim, page, block, T, fmt):
    """Blocks that several warps share, and that do not stay in registers."""
    rng = np.random.default_rng(T + dim)
    lengths = [T - 100, 100]
    table, pages = au.shuffled_table(rng, lengths, page)
    c = au.cache_arrays(rng, fmt, pages, heads, page, dim, block, table)
    dc = au.DeviceCache(G, c)
    seq, pos = np.repeat([0, 1], lengths).astype(np.int32), np.concatenate([np.arange(n) for n in lengths]).astype(np.int32)
    k, v = values(rng, (T, heads, dim), False), values(rng, (T, heads, dim), False)
    for a, b in ((0, 17), (17, T)):  # behind 17 tokens that were there
        G.cache_store(dc.cache, dev_tensor(k[a:b]), dev_tensor(v[a:b]), b - a, dev_tensor(seq[a:b]), dev_tensor(pos[a:b]))
        oatt.store(c, k[a:b], v[a:b], seq[a:b], pos[a:b])
    same_cache(dc, c)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("heads, dim, page, block", [(1, 16, 16, 16), (5, 64, 32, 4), (6, 80, 16, 2), (9, 128, 64, 1), (3, 256, 16, 1),
                                                     (2, 48, 64, 4)])
def test_small_blocks_of_prompts(G, heads, dim, page, block, fmt, f16):
    """Blocks that a warp holds at once, several heads of them; blocks begun before, tokens without a place."""
    rng = np.random.default_rng(3 * dim + block)
    lengths, begun = [270, 1, 98], [3, 0, 7]
    table, pages = au.shuffled_table(rng, lengths, page)
    table[0, 2] = -1
    c = au.cache_arrays(rng, fmt, pages, heads, page, dim, block, table)
    dc = au.DeviceCache(G, c)
    for a, b in ((np.zeros(3, dtype=int), begun), (begun, lengths)):
        seq = np.repeat([0, 1, 5, 2], [b[0] - a[0], b[1] - a[1], 4, b[2] - a[2]]).astype(np.int32)
        pos = np.concatenate([np.arange(a[0], b[0]), np.arange(a[1], b[1]), np.arange(4), np.arange(a[2], b[2])]).astype(np.int32)
        k, v = values(rng, (len(seq), heads, dim), f16), values(rng, (len(seq), heads, dim), f16)
        G.cache_store(dc.cache, dev_tensor(k), dev_tensor(v), len(seq), dev_tensor(seq), dev_tensor(pos), type=fmt_type(G, k))
        oatt.store(c, k, v, seq, pos)
        same_cache(dc, c)


@pytest.mark.parametrize("T", [3, 600])
def test_queries_without_a_place(G, T):
    """Left as they were, among ones that are turned."""
    H, Hq, D, block = 2, 5, 48, 1
    rng = np.random.default_rng(T)
    c = au.cache_arrays(rng, "i8", 40, H, 16, D, block, np.arange(40)[None, :])
    dc = au.DeviceCache(G, c)
    seq, pos = np.where(np.arange(T) % 7 == 2, 1, 0).astype(np.int32), np.arange(T, dtype=np.int32)
    q, k, v = (dev_tensor(values(rng, (T, h, D), False)) for h in (Hq, H, H))
    rot = torch.empty(G.rope_table_bytes(D), dtype=torch.uint8, device="cuda")
    G.rope_table(rot, D)
    want, got = torch.empty_like(q), torch.full_like(q, 7.0)
    G.rope(q, T, Hq, D, dev_tensor(pos), rot, want)
    G.cache_store(dc.cache, k, v, T, dev_tensor(seq), dev_tensor(pos), rope=rot, q=q, q_heads=Hq, q_dst=got)
    want[dev_tensor(seq) == 1] = 7.0
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_hard_values(G, fmt):
    """Ties, zeros, the largest and smallest magnitudes, scales at both ends."""
    rng = np.random.default_rng(7)
    tops = np.array([127.0, 448.0, 0.0, 1e-45, 1e-38, 2.0 ** -105, 3.4028235e38, 3.39e38, 1.0, 127.5, 1e30, 5e-33, 126.99999, 448.00003,
                     0.1, 65504.0], dtype=np.float32)
    n = len(tops)
    c = au.cache_arrays(rng, fmt, 4, 1, 16, 256, 1, [[0, 1, 2]])
    dc = au.DeviceCache(G, c)
    x = np.zeros((n, 1, 256), dtype=np.float32)
    for i, a in enumerate(tops):
        d = oatt.least_scale(fmt, float(a))
        halves = (np.arange(254) - 127 + 0.5) * d if fmt == "i8" else np.concatenate(
            ((oatt.E4M3[:126] + oatt.E4M3[1:127]) / 2, -(oatt.E4M3[:126] + oatt.E4M3[1:127]) / 2, [0, 0])) * d
        x[i, 0, 0] = a
        x[i, 0, 1:255] = np.clip(halves.astype(np.float32), -a, a)  # ties are exact in 32 bits
        x[i, 0, 255] = np.nextafter(x[i, 0, 100], np.float32(-1))
    seq, pos = np.zeros(n, dtype=np.int32), np.arange(n, dtype=np.int32)
    G.cache_store(dc.cache, dev_tensor(x), dev_tensor(-x), n, dev_tensor(seq), dev_tensor(pos))
    oatt.store(c, x, -x, seq, pos)
    assert np.array_equal(dc.host("k_scale"), c["k_scale"]) and np.array_equal(dc.host("v_scale"), c["v_scale"])
    for name in "kv":  # (minus zero is another e4m3 code of the same value)
        assert np.array_equal(oatt.decode(fmt, dc.host(name)), oatt.decode(fmt, c[name]))


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_not_finite(G, fmt):
    rng = np.random.default_rng(8)
    c = au.cache_arrays(rng, fmt, 3, 2, 16, 32, 8, [[2, 0]])
    dc = au.DeviceCache(G, c)
    steps = [(0, 8), (8, 11), (11, 12), (12, 20), (8, 9)]
    for i, (a, b) in enumerate(steps):
        k, v = values(rng, (b - a, 2, 32), False), values(rng, (b - a, 2, 32), False)
        if i == 1:
            k[1, 0, 3], v[2, 1, 31] = np.nan, -np.inf
        seq, pos = np.zeros(b - a, dtype=np.int32), np.arange(a, b, dtype=np.int32)
        G.cache_store(dc.cache, dev_tensor(k), dev_tensor(v), b - a, dev_tensor(seq), dev_tensor(pos))
        oatt.store(c, k, v, seq, pos)
        same_cache(dc, c)
    out = [torch.empty(20, 2, 32, device="cuda") for _ in range(2)]
    seq, pos = np.zeros(20, dtype=np.int32), np.arange(20, dtype=np.int32)
    G.cache_load(dc.cache, 20, dev_tensor(seq), dev_tensor(pos), *out)
    for o, w in zip(out, oatt.load(c, seq, pos)):
        assert np.array_equal(o.double().cpu().numpy(), w, equal_nan=True)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_bad_pages_and_places(G, fmt):
    """Rows without a place change nothing; a table with pages out of range is not followed."""
    rng = np.random.default_rng(9)
    table = [[0, 1 << 30, 2], [-5, 1, 3], [4, 5, 2 ** 31 - 1]]
    c = au.cache_arrays(rng, fmt, 4, 2, 16, 48, 4, table)
    dc = au.DeviceCache(G, c)
    seq = np.array([0, 0, 0, 1, 1, 2, 2, 3, -1, -2 ** 31, 2 ** 31 - 1, 0, 0, 0], dtype=np.int32)
    pos = np.array([15, 16, 32, 0, 16, 0, 16, 0, 0, 0, 0, 48, -1, 2 ** 31 - 1], dtype=np.int32)
    k, v = values(rng, (len(seq), 2, 48), True), values(rng, (len(seq), 2, 48), True)
    G.cache_store(dc.cache, dev_tensor(k), dev_tensor(v), len(seq), dev_tensor(seq), dev_tensor(pos), type=G.F16)
    before = {n: c[n].copy() for n in ("k", "v")}
    oatt.store(c, k, v, seq, pos)
    same_cache(dc, c)
    assert not np.array_equal(c["k"], before["k"])
    out = [torch.full((len(seq), 2, 48), 5.0, device="cuda") for _ in range(2)]
    G.cache_load(dc.cache, len(seq), dev_tensor(seq), dev_tensor(pos), *out)
    for o, w in zip(out, oatt.load(c, seq, pos)):
        assert np.array_equal(o.double().cpu().numpy(), w)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("ld, at", [(0, 0), (300, 0), (257, 3), (260, 4), (320, 2)])
def test_strides_and_alignment(G, ld, at, f16):
    rng = np.random.default_rng(ld + at)
    c = au.cache_arrays(rng, "i8", 5, 2, 16, 128, 4, [[3, 1], [0, 4]])
    dc = au.DeviceCache(G, c)
    seq, pos = np.repeat([0, 1], [20, 9]).astype(np.int32), np.concatenate((np.arange(2, 22), np.arange(9))).astype(np.int32)
    k, v = values(rng, (29, 2, 128), f16), values(rng, (29, 2, 128), f16)
    kt, vt = rows_on(k, ld, at), rows_on(v, 0, at)
    G.cache_store(dc.cache, kt, vt, 29, dev_tensor(seq), dev_tensor(pos), type=fmt_type(G, k), ldk=ld)
    oatt.store(c, k, v, seq, pos)
    same_cache(dc, c)
    w = ld or 256
    out = [torch.full((at + 29 * w + 8,), 7.0, dtype=torch.float16 if f16 else torch.float32, device="cuda") for _ in range(2)]
    G.cache_load(dc.cache, 29, dev_tensor(seq), dev_tensor(pos), out[0][at:], None, type=fmt_type(G, k), ldk=ld)
    G.cache_load(dc.cache, 29, dev_tensor(seq), dev_tensor(pos), None, out[1][at:], type=fmt_type(G, k), ldv=ld)
    for o, want in zip(out, oatt.load(c, seq, pos)):
        rows = o[at:at + 29 * w].view(29, w)
        assert torch.equal(rows[:, :256].cpu(), torch.from_numpy(want.reshape(29, -1).astype(np.float32)).to(o.dtype))
        assert torch.all(rows[:, 256:] == 7.0) and torch.all(o[:at] == 7.0) and torch.all(o[at + 29 * w:] == 7.0)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("T, dim, n_rot, block, fused", [(5, 128, 128, 16, True), (1, 64, 32, 1, False), (300, 128, 64, 32, True),
                                                         (40, 80, 40, 4, False), (270, 256, 256, 64, False), (3, 96, 0, 16, True),
                                                         (290, 128, 64, 2, True), (400, 80, 0, 1, False)])
def test_with_rotation(G, T, dim, n_rot, block, fused, layout, f16):
    """Equal, bit for bit, to gf_rope followed by the store of its 32-bit results; queries to gf_rope's."""
    rng = np.random.default_rng(T + dim)
    H, Hq, page = 2, 6, 64
    before = 11
    table, pages = au.shuffled_table(rng, [before + T], page)
    c = au.cache_arrays(rng, "i8", pages, H, page, dim, block, table)
    a, b = au.DeviceCache(G, c), au.DeviceCache(G, c)
    dt = torch.float16 if f16 else torch.float32
    typ = G.F16 if f16 else G.F32
    seq, pos = dev_tensor(np.zeros(T, dtype=np.int32)), dev_tensor(np.arange(before, before + T, dtype=np.int32))
    rot = torch.empty(G.rope_table_bytes(n_rot or dim), dtype=torch.uint8, device="cuda")
    G.rope_table(rot, n_rot or dim)
    x = dev_tensor(values(rng, (T, Hq + 2 * H, dim), f16))
    q, k, v = x[:, :Hq].contiguous(), x[:, Hq:Hq + H].contiguous(), x[:, Hq + H:].contiguous()
    kr = torch.empty(T, H, dim, device="cuda")
    G.rope(k.float(), T, H, dim, pos, rot, kr, n_rot=n_rot, layout=layout)
    G.cache_store(b.cache, kr, v.float(), T, seq, pos)
    qr = torch.empty_like(q)
    G.rope(q, T, Hq, dim, pos, rot, qr, n_rot=n_rot, layout=layout, type=typ)
    kw = dict(type=typ, rope=rot, n_rot=n_rot, layout=layout, q_heads=Hq)
    if fused:  # one buffer of q, k, v rows, queries turned in place
        y, ld = x.clone().reshape(T, -1), (Hq + 2 * H) * dim
        flat = y.reshape(-1)
        G.cache_store(a.cache, flat[Hq * dim:], flat[(Hq + H) * dim:], T, seq, pos, ldk=ld, ldv=ld, q=y, q_dst=y, ldq=ld,
                      ld_q_dst=ld, **kw)
        got = y.view(T, -1, dim)
        assert torch.equal(got[:, Hq:], x[:, Hq:])
        got = got[:, :Hq]
    else:
        got = torch.zeros_like(q)
        G.Graph([G.prepare_cache_store(a.cache, k, v, T, seq, pos, q=q, q_dst=got, **kw)]).launch()
    assert torch.equal(got, qr)
    for name in ("k_scale", "v_scale", "k", "v"):
        assert np.array_equal(a.host(name), b.host(name)), name
    oatt.store(c, kr.cpu().numpy(), v.float().cpu().numpy(), np.zeros(T, dtype=int), np.arange(before, before + T))
    same_cache(a, c)


def test_far_into_a_large_pool(G):
    """Code offsets beyond 32 bits."""
    H, page, D, block = 8, 64, 128, 16
    n_pages = (5 << 30) // (H * page * D)
    k, v = (torch.zeros(n_pages * H * page * D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n_pages * H * (page // block), device="cuda") for _ in range(2))
    table = dev_tensor(np.array([[n_pages - 1, 3]], dtype=np.int32))
    cache = G.Cache(k, v, ks, vs, G.CACHE_I8, n_pages, H, page, D, block, table, 1, 2)
    x = torch.randn(70, H, D, device="cuda")
    seq, pos = torch.zeros(70, dtype=torch.int32, device="cuda"), torch.arange(70, dtype=torch.int32, device="cuda")
    G.cache_store(cache, x, -x, 70, seq, pos)
    a, b = torch.empty_like(x), torch.empty_like(x)
    G.cache_load(cache, 70, seq, pos, a, b)
    assert torch.equal(a, -b) and float((a - x).abs().max()) <= 0.51 * float(x.abs().max()) / 127 * 1.001
    used = torch.zeros(n_pages, dtype=torch.bool, device="cuda")
    used[n_pages - 1] = used[3] = True
    assert not bool(k.view(n_pages, -1).any(1)[~used].any()) and not bool(ks.view(n_pages, -1).any(1)[~used].any())
