"""Argument checks of gf_rope, gf_cache_store, gf_cache_load and gf_attend that need no GPU: every refusal
comes before a launch.  Pointers are fake, well-separated device addresses."""

import ctypes

import pytest

X, DST, POS, SEQ, TAB, Q, QD = [(i << 40) for i in range(1, 8)]
K, V, KS, VS, PT, WS, LSE, NK, NV = [(i << 40) for i in range(8, 17)]
BIG = 1 << 36


def cache(lib, **kw):
    d = dict(k=K, v=V, k_scale=KS, v_scale=VS, format=0, n_pages=10, heads=2, page=16, dim=64, block=16, table=PT, n_seqs=3,
             table_ld=4)
    d.update(kw)
    return lib.Cache(**d)


CACHE = [
    (dict(format=2), "INVALID"), (dict(n_pages=-1), "INVALID"), (dict(heads=0), "INVALID"), (dict(dim=0), "INVALID"),
    (dict(page=0), "INVALID"), (dict(page=24), "INVALID"), (dict(block=0), "INVALID"), (dict(block=3), "INVALID"),
    (dict(block=32), "INVALID"), (dict(n_seqs=-1), "INVALID"), (dict(table_ld=-1), "INVALID"),
    (dict(page=8, block=8), "UNSUPPORTED"), (dict(page=128, block=128), "UNSUPPORTED"), (dict(dim=24), "UNSUPPORTED"),
    (dict(dim=272), "UNSUPPORTED"), (dict(heads=1025), "UNSUPPORTED"), (dict(page=1 << 21), "UNSUPPORTED"),
    (dict(table_ld=1 << 27), "UNSUPPORTED"), (dict(n_pages=1 << 31), "UNSUPPORTED"),
    (dict(n_pages=(1 << 31) - 1, heads=1024, page=1 << 20), "UNSUPPORTED"),
    (dict(k=None), "INVALID"), (dict(v=None), "INVALID"), (dict(k_scale=None), "INVALID"), (dict(v_scale=None), "INVALID"),
    (dict(table=None), "INVALID"), (dict(k=K + 8), "ALIGN"), (dict(v=V + 1), "ALIGN"), (dict(k_scale=KS + 2), "ALIGN"),
    (dict(v_scale=VS + 1), "ALIGN"), (dict(table=PT + 2), "ALIGN"),
    (dict(v=K), "ALIAS"), (dict(k_scale=K + 64), "ALIAS"), (dict(v_scale=KS), "ALIAS"), (dict(table=V + 16), "ALIAS"),
]


def rope(lib, T=2, H=3, D=64, x=X, dst=DST, pos=POS, table=TAB, **kw):
    return lib.rope(x, T, H, D, pos, table, dst, check=False, stream=0, **kw)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), "INVALID"), (dict(H=-1), "INVALID"), (dict(D=1), "INVALID"), (dict(type=2), "INVALID"),
    (dict(n_rot=3), "INVALID"), (dict(n_rot=66), "INVALID"), (dict(n_rot=-2), "INVALID"), (dict(layout=2), "INVALID"),
    (dict(D=63), "INVALID"), (dict(T=(1 << 20) + 1), "UNSUPPORTED"), (dict(H=1025), "UNSUPPORTED"), (dict(D=1026), "UNSUPPORTED"),
    (dict(ld=191), "INVALID"), (dict(ld_dst=100), "INVALID"), (dict(ld=1 << 41), "UNSUPPORTED"),
    (dict(x=None), "INVALID"), (dict(dst=None), "INVALID"), (dict(pos=None), "INVALID"), (dict(table=None), "INVALID"),
    (dict(x=X + 2), "ALIGN"), (dict(dst=DST + 1, type=1), "ALIGN"), (dict(pos=POS + 2), "ALIGN"), (dict(table=TAB + 8), "ALIGN"),
    (dict(dst=X + 4), "ALIAS"), (dict(dst=X, ld_dst=200), "ALIAS"), (dict(dst=POS - 16), "ALIAS"), (dict(dst=TAB), "ALIAS"),
    (dict(dst=TAB + 16 + 31 * 8, D=64), "ALIAS"),
])
def test_rope_refusals(lib, kw, want):
    assert rope(lib, **kw) == getattr(lib, "ERR_" + want)


def test_nothing_to_do(lib):
    assert rope(lib, T=0, x=None, dst=None) == lib.OK and rope(lib, H=0) == lib.OK
    assert store(lib, T=0, k=None, v=None, pos=None) == lib.OK
    assert load(lib, T=0) == lib.OK and load(lib, k=None, v=None) == lib.OK
    assert att(lib, T=0, q=None, ws=None) == lib.OK
    h = ctypes.c_void_p(7)
    assert lib.raw.gf_prepare_attend(None, Q, 1, 2, SEQ, POS, None, DST, ctypes.byref(h)) == lib.ERR_INVALID and not h.value
    assert lib.raw.gf_prepare_rope(X, 1, 1, 64, POS, None, DST, None) == lib.ERR_INVALID
    assert lib.raw.gf_cache_store(None, K, V, 1, SEQ, POS, None, None) == lib.ERR_INVALID
    assert lib.raw.gf_cache_load(None, 1, SEQ, POS, None, K, V, None) == lib.ERR_INVALID


@pytest.mark.parametrize("kw, want", [
    (dict(n_rot=0), "INVALID"), (dict(n_rot=7), "INVALID"), (dict(n_rot=1026), "UNSUPPORTED"), (dict(kind=4), "INVALID"),
    (dict(base=1.0), "INVALID"), (dict(base=float("inf")), "INVALID"), (dict(magnitude=-1.0), "INVALID"),
    (dict(kind=1, factor=0.0), "INVALID"), (dict(kind=2, factor=2.0), "INVALID"), (dict(kind=3, factor=2.0, span=0), "INVALID"),
    (dict(kind=2, factor=2.0, span=8192, fast=1.0, slow=1.0), "INVALID"), (dict(kind=3, factor=2.0, span=8192, slow=0.0), "INVALID"),
    (dict(kind=1, factor=float("nan")), "INVALID"), (dict(table=None), "INVALID"), (dict(table=TAB + 8), "ALIGN"),
    (dict(divisors=X + 2), "ALIGN"), (dict(divisors=TAB + 32), "ALIAS"),
])
def test_rope_table_refusals(lib, kw, want):
    kw = dict(dict(table=TAB, n_rot=64), **kw)
    assert lib.rope_table(kw.pop("table"), kw.pop("n_rot"), check=False, stream=0, **kw) == getattr(lib, "ERR_" + want)


def test_rope_table_bytes(lib):
    assert lib.rope_table_bytes(2) == 24 and lib.rope_table_bytes(128) == 16 + 64 * 8
    for bad in (0, 3, -2, 1026):
        with pytest.raises(lib.GemvFuseError):
            lib.rope_table_bytes(bad)


def store(lib, T=4, k=NK, v=NV, seq=SEQ, pos=POS, c=None, **kw):
    return lib.cache_store(cache(lib, **(c or {})), k, v, T, seq, pos, check=False, stream=0, **kw)


R = dict(rope=TAB, q=Q, q_dst=QD, q_heads=4)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), "INVALID"), (dict(type=3), "INVALID"), (dict(T=(1 << 20) + 1), "UNSUPPORTED"), (dict(q_heads=-1), "INVALID"),
    (dict(k=None), "INVALID"), (dict(v=None), "INVALID"), (dict(pos=None), "INVALID"), (dict(ldk=100), "INVALID"),
    (dict(ldv=127), "INVALID"), (dict(k=NK + 2), "ALIGN"), (dict(v=NV + 1, type=1), "ALIGN"), (dict(seq=SEQ + 2), "ALIGN"),
    (dict(pos=POS + 1), "ALIGN"), (dict(k=K), "ALIAS"), (dict(v=VS), "ALIAS"), (dict(seq=KS), "ALIAS"), (dict(pos=V + 64), "ALIAS"),
    (dict(q=Q, q_dst=QD, q_heads=4), "INVALID"),  # queries without a rotation
    (dict(R, n_rot=20), "UNSUPPORTED"), (dict(R, n_rot=72), "INVALID"), (dict(R, layout=5), "INVALID"),
    (dict(R, rope=TAB + 4), "ALIGN"), (dict(R, rope=K), "ALIAS"), (dict(R, q=None), "INVALID"), (dict(R, q_dst=None), "INVALID"),
    (dict(R, q_heads=1025), "UNSUPPORTED"), (dict(R, ldq=255), "INVALID"), (dict(R, q=Q + 2), "ALIGN"),
    (dict(R, q_dst=Q + 4), "ALIAS"), (dict(R, q_dst=Q, ld_q_dst=300), "ALIAS"), (dict(R, q_dst=NK), "ALIAS"),
    (dict(R, q_dst=K), "ALIAS"), (dict(R, q_dst=TAB), "ALIAS"), (dict(R, q_dst=POS), "ALIAS"), (dict(R, q_dst=PT), "ALIAS"),
    (dict(R, q=V), "ALIAS"),
    # one fused buffer [q | k | v]: the heads of q reach into k
    (dict(R, q=NK, q_dst=NK, ldq=512, ld_q_dst=512, k=NK + 4 * 255, ldk=512, v=NK + 4 * 384, ldv=512), "ALIAS"),
    (dict(R, q=NK, q_dst=NK, ldq=512, ld_q_dst=512, k=NK + 4 * 256, ldk=640, v=NK + 4 * 384, ldv=512), "ALIAS"),
])
def test_store_refusals(lib, kw, want):
    assert store(lib, **kw) == getattr(lib, "ERR_" + want)


def load(lib, T=4, k=NK, v=NV, seq=SEQ, pos=POS, c=None, **kw):
    return lib.cache_load(cache(lib, **(c or {})), T, seq, pos, k, v, check=False, stream=0, **kw)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), "INVALID"), (dict(type=2), "INVALID"), (dict(T=(1 << 20) + 1), "UNSUPPORTED"), (dict(pos=None), "INVALID"),
    (dict(ldk=64), "INVALID"), (dict(k=NK + 1), "ALIGN"), (dict(seq=SEQ + 1), "ALIGN"), (dict(k=K + 64), "ALIAS"),
    (dict(v=NK), "ALIAS"), (dict(k=SEQ), "ALIAS"), (dict(v=POS - 16), "ALIAS"), (dict(v=PT), "ALIAS"), (dict(k=VS), "ALIAS"),
])
def test_load_refusals(lib, kw, want):
    assert load(lib, **kw) == getattr(lib, "ERR_" + want)


def att(lib, T=4, Hq=8, q=Q, seq=SEQ, pos=POS, dst=DST, ws=WS, nbytes=BIG, c=None, **kw):
    return lib.attend(cache(lib, **(c or {})), q, T, Hq, seq, pos, dst, ws, workspace_bytes=nbytes, check=False, stream=0, **kw)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), "INVALID"), (dict(Hq=0), "INVALID"), (dict(Hq=7), "INVALID"), (dict(type=2), "INVALID"), (dict(run=-1), "INVALID"),
    (dict(window=-1), "INVALID"), (dict(scale=-1.0), "INVALID"), (dict(scale=float("nan")), "INVALID"),
    (dict(scale=float("inf")), "INVALID"), (dict(T=(1 << 16) + 1), "UNSUPPORTED"), (dict(Hq=1026), "UNSUPPORTED"),
    (dict(window=1 << 31), "UNSUPPORTED"), (dict(run=(1 << 16) + 1), "UNSUPPORTED"),
    (dict(q=None), "INVALID"), (dict(dst=None), "INVALID"), (dict(pos=None), "INVALID"), (dict(ws=None), "INVALID"),
    (dict(nbytes=1000), "INVALID"), (dict(ldq=511), "INVALID"), (dict(ld_dst=500), "INVALID"),
    (dict(q=Q + 2), "ALIGN"), (dict(dst=DST + 1, type=1), "ALIGN"), (dict(ws=WS + 128), "ALIGN"), (dict(lse=LSE + 2), "ALIGN"),
    (dict(seq=SEQ + 2), "ALIGN"), (dict(dst=Q), "ALIAS"), (dict(dst=K), "ALIAS"), (dict(dst=PT), "ALIAS"), (dict(dst=POS), "ALIAS"),
    (dict(lse=DST), "ALIAS"), (dict(lse=Q + 16), "ALIAS"), (dict(ws=DST), "ALIAS"), (dict(ws=V), "ALIAS"), (dict(q=WS + 256), "ALIAS"),
    (dict(lse=WS + 256), "ALIAS"), (dict(seq=DST), "ALIAS"),
])
def test_attend_refusals(lib, kw, want):
    assert att(lib, **kw) == getattr(lib, "ERR_" + want)


@pytest.mark.parametrize("kw, want", CACHE)
def test_cache_refusals(lib, kw, want):
    e = getattr(lib, "ERR_" + want)
    assert store(lib, c=kw) == e and load(lib, c=kw) == e and att(lib, Hq=kw.get("heads", 2) * 2, c=kw) in (e, lib.ERR_INVALID)


def test_attend_workspace(lib):
    need = lib.attend_workspace(4, 8, 2, 64)
    assert att(lib, nbytes=need - 1) == lib.ERR_INVALID and need < lib.attend_workspace(4, 8, 2, 128)
    for bad in ((-1, 8, 2, 64), (4, 7, 2, 64), (4, 8, 0, 64), (4, 8, 2, 40), (4, 8, 2, 512), (1 << 17, 8, 2, 64), (4, 8, 2, 64, -1)):
        with pytest.raises(lib.GemvFuseError):
            lib.attend_workspace(*bad)
