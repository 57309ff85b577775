"""Argument checks of gf_route, gemv_experts and gemv_lora that need no GPU: every refusal
comes before a launch.  Pointers are fake, well-separated device addresses."""

import ctypes

import pytest

L, I, WT, B = (1 << 40), (2 << 40), (3 << 40), (4 << 40)
G, U, D, X, DST, WS = (5 << 40), (6 << 40), (7 << 40), (8 << 40), (9 << 40), (10 << 40)
BIG = 1 << 36


def r(lib, T=4, E=16, k=2, logits=L, ids=I, w=WT, **kw):
    return lib.route(logits, T, E, k, ids, w, check=False, stream=0, **kw)


@pytest.mark.parametrize("kw, want", [
    (dict(E=0), "INVALID"), (dict(k=0), "INVALID"), (dict(k=17), "INVALID"), (dict(T=-1), "INVALID"),
    (dict(score=2), "INVALID"), (dict(scale=float("nan")), "INVALID"), (dict(scale=float("inf")), "INVALID"),
    (dict(ld=15), "INVALID"), (dict(n_group=3), "INVALID"), (dict(n_group=-2), "INVALID"),
    (dict(n_group=4, topk_group=5), "INVALID"), (dict(n_group=4, topk_group=0), "INVALID"),
    (dict(n_group=4, topk_group=2, group_top=3), "INVALID"),
    (dict(E=1025), "UNSUPPORTED"), (dict(E=64, k=33), "UNSUPPORTED"),
    (dict(E=128, n_group=64, topk_group=2), "UNSUPPORTED"), (dict(T=1 << 25), "UNSUPPORTED"),
    (dict(logits=None), "INVALID"), (dict(ids=None), "INVALID"), (dict(w=None), "INVALID"),
    (dict(logits=L + 2), "ALIGN"), (dict(ids=I + 1), "ALIGN"), (dict(w=WT + 2), "ALIGN"), (dict(bias=B + 2), "ALIGN"),
    (dict(ids=L + 4), "ALIAS"), (dict(w=L), "ALIAS"), (dict(w=I + 16), "ALIAS"), (dict(bias=I), "ALIAS"),
    (dict(ids=L + 4 * 20 * 3 + 60, ld=20), "ALIAS"),
])
def test_route_refusals(lib, kw, want):
    assert r(lib, **kw) == getattr(lib, "ERR_" + want)


def test_route_nothing_to_do(lib):
    assert r(lib, T=0) == lib.OK
    assert r(lib, T=0, logits=None, ids=None, w=None) == lib.OK


def test_route_null_options(lib):
    assert lib.raw.gf_route(L, 1, 8, None, I, WT, None) == lib.ERR_INVALID
    h = ctypes.c_void_p(7)
    assert lib.raw.gf_prepare_route(L, 1, 8, None, I, WT, ctypes.byref(h)) == lib.ERR_INVALID and not h.value
    assert lib.raw.gf_prepare_route(L, 1, 8, None, I, WT, None) == lib.ERR_INVALID


def e(lib, T=2, E=4, k=2, M=64, K=128, wt=3, wd=3, gate=G, up=U, down=D, x=X, ids=I, w=WT, aux=None, dst=DST, ws=WS,
      nbytes=BIG, norm=None, eps=1e-6):
    return lib.gemv_experts(gate, up, wt, down, wd, E, x, M, K, ids, w, T, k, aux, dst, ws, workspace_bytes=nbytes,
                            rms_norm_weight=norm, rms_norm_eps=eps, check=False, stream=0)


@pytest.mark.parametrize("kw, want", [
    (dict(wt=5), "INVALID"), (dict(wd=-1), "INVALID"), (dict(E=0), "INVALID"), (dict(k=0), "INVALID"),
    (dict(T=-1), "INVALID"), (dict(M=-32), "INVALID"), (dict(K=-32), "INVALID"),
    (dict(T=257), "UNSUPPORTED"), (dict(E=1025), "UNSUPPORTED"), (dict(k=33), "UNSUPPORTED"),
    (dict(K=100), "UNSUPPORTED"), (dict(M=40), "UNSUPPORTED"), (dict(wt=4), "UNSUPPORTED"), (dict(wd=4), "UNSUPPORTED"),
    (dict(K=1 << 21), "UNSUPPORTED"),
    (dict(gate=None), "INVALID"), (dict(up=None), "INVALID"), (dict(down=None), "INVALID"), (dict(x=None), "INVALID"),
    (dict(ids=None), "INVALID"), (dict(w=None), "INVALID"), (dict(dst=None), "INVALID"), (dict(ws=None), "INVALID"),
    (dict(nbytes=1000), "INVALID"),
    (dict(gate=G + 1), "ALIGN"), (dict(x=X + 2), "ALIGN"), (dict(dst=DST + 2), "ALIGN"), (dict(ws=WS + 128), "ALIGN"),
    (dict(ids=I + 2), "ALIGN"), (dict(w=WT + 1), "ALIGN"), (dict(aux=B + 2), "ALIGN"), (dict(down=D + 1), "ALIGN"),
    (dict(dst=X), "ALIAS"), (dict(dst=G + 16), "ALIAS"), (dict(dst=U), "ALIAS"), (dict(dst=D), "ALIAS"),
    (dict(dst=I), "ALIAS"), (dict(dst=WT), "ALIAS"), (dict(aux=DST + 4), "ALIAS"), (dict(ws=X), "ALIAS"),
    (dict(norm=B + 2), "ALIGN"), (dict(norm=B, eps=-1.0), "INVALID"), (dict(norm=B, eps=float("nan")), "INVALID"),
    (dict(norm=DST), "ALIAS"), (dict(norm=WS + 64), "ALIAS"),
    (dict(dst=WS + 256), "ALIAS"), (dict(aux=WS), "ALIAS"), (dict(ids=WS + 4), "ALIAS"), (dict(gate=WS + 1024), "ALIAS"),
])
def test_experts_refusals(lib, kw, want):
    assert e(lib, **kw) == getattr(lib, "ERR_" + want)


def test_experts_nothing_to_do(lib):
    assert e(lib, T=0) == lib.OK
    assert e(lib, K=0) == lib.OK


def test_experts_workspace(lib):
    assert lib.experts_workspace(4, 0, 2, 64, 128) >= 0
    small, large = lib.experts_workspace(128, 1, 8, 768, 2048), lib.experts_workspace(128, 256, 8, 768, 2048)
    assert 0 < small < large
    assert e(lib, nbytes=lib.experts_workspace(4, 2, 2, 64, 128) - 1) == lib.ERR_INVALID
    for bad in ((0, 1, 1, 1, 1), (1, -1, 1, 1, 1), (1, 1, 0, 1, 1), (1, 257, 1, 1, 1)):
        with pytest.raises(lib.GemvFuseError):
            lib.experts_workspace(*bad)


def lo(lib, N=2, M=64, K=128, wt=3, epi=0, W=G, x=X, aux=None, dst=DST, A=U, Bm=D, at=1, n=3, rank=8, ids=I, s=None,
       ws=WS, nbytes=BIG, **opts):
    return lib.gemv_lora(W, wt, x, M, K, epi, aux, dst, A, Bm, at, n, rank, ids, s, ws, workspace_bytes=nbytes,
                         check=False, stream=0, ncols=N, **opts)


@pytest.mark.parametrize("kw, want", [
    (dict(at=2), "INVALID"), (dict(n=-1), "INVALID"), (dict(rank=0), "INVALID"), (dict(rank=257), "UNSUPPORTED"),
    (dict(N=-1), "INVALID"), (dict(N=257), "UNSUPPORTED"), (dict(K=100), "UNSUPPORTED"), (dict(epi=5), "INVALID"),
    (dict(epi=4), "INVALID"), (dict(W=None), "INVALID"), (dict(x=None), "INVALID"), (dict(A=None), "INVALID"),
    (dict(Bm=None), "INVALID"), (dict(ids=None), "INVALID"), (dict(ws=None), "INVALID"), (dict(nbytes=100), "INVALID"),
    (dict(fwht_signs=B, fwht_block=64, nsigns=64), "UNSUPPORTED"),
    (dict(A=U + 1), "ALIGN"), (dict(at=0, Bm=D + 2), "ALIGN"), (dict(ids=I + 2), "ALIGN"), (dict(s=WT + 2), "ALIGN"),
    (dict(ws=WS + 64), "ALIGN"),
    (dict(dst=U), "ALIAS"), (dict(dst=D + 2 * 64 * 8), "ALIAS"), (dict(dst=I + 4), "ALIAS"), (dict(s=DST), "ALIAS"),
    (dict(dst=G), "ALIAS"), (dict(dst=X), "ALIAS"), (dict(dst=WS), "ALIAS"), (dict(x=WS), "ALIAS"),
    (dict(W=WS + 256), "ALIAS"), (dict(A=WS), "ALIAS"), (dict(epi=4, aux=WS + 256), "ALIAS"),
    (dict(epi=4, aux=DST + 4), "ALIAS"),
])
def test_lora_refusals(lib, kw, want):
    assert lo(lib, **kw) == getattr(lib, "ERR_" + want)


def test_lora_nothing_to_do(lib):
    assert lo(lib, M=0) == lib.OK


def test_lora_workspace(lib):
    assert lib.lora_workspace(1, 4096, 4096, 16, 8) < lib.lora_workspace(8, 4096, 4096, 16, 8)
    assert lo(lib, nbytes=lib.lora_workspace(2, 64, 128, 8, 3) - 1) == lib.ERR_INVALID
    for bad in ((-1, 1, 1, 1, 1), (1, 1, 1, 0, 1), (257, 1, 1, 1, 1), (1, 1, 1, 257, 1)):
        with pytest.raises(lib.GemvFuseError):
            lib.lora_workspace(*bad)
