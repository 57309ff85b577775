"""The attention block's step: q, k, v products, rotation, cache, attention and output projection in one graph,
each stage against the fp64 oracle on the stage's own inputs, over several steps."""

import numpy as np
import pytest

import attend_util as au
from decode_gemv_epilogue_gb300 import synth
from gpu_util import TOL_NORM_REL, assert_within
from oracle import attend as oatt
from oracle import gemv as ogemv
from oracle import norm as onorm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def products(s, h, n, name, M, K, extra):
    want = ogemv.gemv(h[name], s.wtype, n, M, K)
    return want, (2e-5 + extra) * ogemv.abs_dot(h[name], s.wtype, n, M, K) + 1e-6


# T, d, heads, kv heads, dim, sequences, tokens of a sequence next to each other
@pytest.mark.parametrize("T, d, H, KV, D, S, run, wt, fmt", [(1, 512, 4, 1, 64, 1, 1, synth.Q4_0, 0), (5, 256, 4, 2, 128, 5, 1, synth.Q8_0, 1),
                                                           (12, 256, 8, 2, 32, 4, 3, synth.F16, 0)])
def test_steps(lib, T, d, H, KV, D, S, run, wt, fmt):
    from decode_gemv_epilogue_gb300.attn_step import AttnStep
    s = AttnStep(T, d, H, KV, D, S, 100, wtype=wt, fmt=fmt, page=16, block=4, run=run, seed=T)
    c = dict(fmt="i8" if fmt == 0 else "e4m3", block=4, k=s.k.cpu().numpy(), v=s.v.cpu().numpy(),
             k_scale=s.k_scale.cpu().numpy(), v_scale=s.v_scale.cpu().numpy(), table=s.table.cpu().numpy())
    h, f = s.host, oatt.freqs(D)
    side = torch.cuda.Stream()
    for step in range(20):
        x = synth.normal(T * d, seed=100 + step).astype(np.float32).reshape(T, d)
        seq = np.repeat(np.arange(S), run).astype(np.int32)
        pos = (step * run + np.tile(np.arange(run), S)).astype(np.int32)
        if step == 7 and T > 1:
            seq[-run:] = -1  # a request that has ended: its rows are padding
        for dst, src in ((s.x, x), (s.seq, seq), (s.pos, pos)):
            dst.copy_(torch.from_numpy(src))
        torch.cuda.synchronize()
        s.launch(stream=side)
        side.synchronize()
        q, k, v, o, y = (getattr(s, n).cpu().numpy() for n in ("q", "new_k", "new_v", "o", "y"))
        live = seq >= 0
        n = onorm.rms_norm(x, h["gamma"], s.eps, d)
        for name, got, heads in (("wk", k, KV), ("wv", v, KV)):
            want, b = products(s, h, n, name, heads * D, d, TOL_NORM_REL)
            assert_within(got.reshape(T, -1), want, b, name)
        # queries: a rotation keeps a pair's size, its own rounding is 2^-20 of it
        want, b = products(s, h, n, "wq", H * D, d, TOL_NORM_REL)
        want = np.where(live[:, None, None], oatt.rope(want.reshape(T, H, D), pos, f), want.reshape(T, H, D))
        b = b.reshape(T, H, D)
        b = b + np.concatenate((b[..., D // 2:], b[..., :D // 2]), -1) + 2.0 ** -19 * np.abs(want).max(-1, keepdims=True)
        assert_within(q, want, b, "q")
        # the cache: the oracle's codes for the oracle's rotation of the kernel's k; a rotation's rounding may turn a
        # code that lies on an edge (2^-20 of the values near one), never by more than one step
        oatt.store(c, oatt.rope(k, pos, f), v, seq, pos)
        for m in "kv":
            got, sc = getattr(s, m).cpu().numpy(), getattr(s, m + "_scale").cpu().numpy()
            a = oatt.decode(c["fmt"], got) * sc.repeat(4, -1)[..., None]
            w = oatt.decode(c["fmt"], c[m]) * c[m + "_scale"].repeat(4, -1)[..., None]
            d_ = np.maximum(sc, c[m + "_scale"]).repeat(4, -1)[..., None]
            # (a value at an edge of the scales themselves: the next power of two, with e4m3)
            assert np.all(np.abs(a - w) <= (1.01 * d_ if fmt == 0 else np.abs(w) / 8 * 1.01 + d_)) and np.mean(a != w) < 1e-2
            c[m], c[m + "_scale"] = got.copy(), sc.copy()
        want, lse, mass, spread = oatt.attend(c, q, seq, pos)
        keys = np.repeat(np.where(live, pos + 1.0, 0.0)[:, None], H, 1)
        b, _ = au.attend_bounds(c, want, lse, mass, spread, keys, False)
        assert_within(o, want, b, "attention")
        want = ogemv.gemv(h["wo"], wt, o.reshape(T, -1), d, H * D, ogemv.EPI_ADD, x)
        assert_within(y, want, 2e-5 * ogemv.abs_dot(h["wo"], wt, o.reshape(T, -1), d, H * D) + 1e-6 + 1e-6 * np.abs(want), "projection")
    assert lib.device_status() == 0
