"""Guard bands around every operand of rotary positions, the 8-bit cache and attention: 4 KiB of a known byte
before and behind each, untouched after calls on ragged shapes; the outputs are checked too, so that no band stays
clean because nothing was written."""

import numpy as np
import pytest

import attend_util as au
from gpu_util import assert_within
from oracle import attend as oatt

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import test_gpu_redzone as rz  # noqa: E402
from test_gpu_redzone_select import Guarded  # noqa: E402


@pytest.fixture(scope="module")
def G(lib):
    assert lib.device_status(reset=True) == 0
    yield lib
    assert lib.device_status() == 0


@pytest.mark.parametrize("T, H, D, n_rot, ld, at", [(1, 1, 2, 2, 0, 0), (3, 5, 7, 4, 40, 4), (37, 25, 80, 40, 0, 0), (300, 3, 128, 128, 400, 16),
                                                    (5, 40, 64, 64, 0, 8)])
def test_rope(G, T, H, D, n_rot, ld, at):
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, ld or H * D)).astype(np.float32)
    pos = rng.integers(0, 9000, T).astype(np.int32)
    X, P = Guarded(x.reshape(-1)[:(T - 1) * (ld or H * D) + H * D], at=at), Guarded(pos, at=4)
    R, Y = Guarded(n=G.rope_table_bytes(n_rot), dtype=torch.uint8, at=16), Guarded(n=T * H * D, at=at)
    G.rope_table(R.t, n_rot)
    for layout in (0, 1):
        G.rope(X.t, T, H, D, P.t, R.t, Y.t, n_rot=n_rot, layout=layout, ld=ld)
        rz.check_all(X, P, R, Y)
        xs = x[:, :H * D].reshape(T, H, D).astype(np.float64)
        want = oatt.rope(xs, pos, oatt.freqs(n_rot), layout=("halves", "pairs")[layout])
        assert np.all(np.abs(Y.t.view(T, H, D).cpu().numpy() - want) <= 2.0 ** -19 * np.abs(xs).max(-1, keepdims=True) + 1e-30)


# heads, group, dim, page, block, lengths, tokens of each
CASES = [(1, 1, 16, 16, 1, [1], 1), (2, 4, 64, 16, 4, [33, 7, 100], 1), (3, 5, 80, 32, 32, [65, 31], 2), (2, 2, 128, 64, 16, [1, 129, 64, 63], 3),
         (1, 16, 128, 16, 2, [300, 5], 5), (2, 3, 256, 64, 64, [70, 128, 2], 1), (1, 9, 192, 16, 16, [47], 4), (1, 33, 48, 32, 8, [64, 90], 1)]


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("H, group, D, page, block, lengths, per", CASES)
def test_store_load_attend(G, H, group, D, page, block, lengths, per, f16, fmt):
    rng = np.random.default_rng(D + H)
    per = min(per, min(lengths))
    table, pages = au.shuffled_table(rng, lengths, page, spare=0)
    c = au.cache_arrays(rng, fmt, pages, H, page, D, block, table)
    a = {k: Guarded(c[k], at=16) for k in ("k", "v", "k_scale", "v_scale", "table")}
    cache = G.Cache(a["k"].t, a["v"].t, a["k_scale"].t, a["v_scale"].t, G.CACHE_I8 if fmt == "i8" else G.CACHE_E4M3, pages, H, page, D,
                    block, a["table"].t, len(lengths), table.shape[1])
    dt, typ, np_t = (torch.float16, G.F16, np.float16) if f16 else (torch.float32, G.F32, np.float32)
    seq, pos = au.positions(lengths, per)
    T, Hq = len(seq), H * group
    S, P = Guarded(seq, at=4), Guarded(pos, at=8)
    k, v, q = (rng.standard_normal((T, h, D)).astype(np_t) for h in (H, H, Hq))
    for at in (0, 2 if f16 else 4):
        K, V, Q = (Guarded(x, at=at) for x in (k, v, q))
        Y, L = Guarded(n=T * Hq * D, dtype=dt, at=at), Guarded(n=T * Hq, at=4)
        BK, BV = (Guarded(n=T * H * D, dtype=dt, at=at) for _ in range(2))
        W = Guarded(n=G.attend_workspace(T, Hq, H, D, per), dtype=torch.uint8)
        every = [*a.values(), S, P, K, V, Q, Y, L, BK, BV, W]
        G.cache_store(cache, K.t, V.t, T, S.t, P.t, type=typ)
        G.cache_load(cache, T, S.t, P.t, BK.t, BV.t, type=typ)
        G.attend(cache, Q.t, T, Hq, S.t, P.t, Y.t, W.t, type=typ, run=per, lse=L.t)
        rz.check_all(*every)
        oatt.store(c, k, v, seq, pos)
        for n in ("k", "v", "k_scale", "v_scale"):
            assert np.array_equal(a[n].t.cpu().numpy().reshape(c[n].shape), c[n]), n
        for got, want in zip((BK, BV), oatt.load(c, seq, pos)):
            assert torch.equal(got.t.cpu(), torch.from_numpy(want.reshape(-1).astype(np.float32)).to(dt))
        want, lse, mass, spread = oatt.attend(c, q, seq, pos)
        b, bl = au.attend_bounds(c, want, lse, mass, spread, np.repeat(pos[:, None] + 1.0, Hq, 1), f16)
        assert_within(Y.t.view(T, Hq, D).double().cpu().numpy(), want, b, "out")
        assert_within(L.t.view(T, Hq).double().cpu().numpy(), lse, bl, "lse")
