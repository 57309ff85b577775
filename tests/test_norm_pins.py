"""The norm-wise check of the experts' product: it refuses what the elementwise bound lets pass."""

import numpy as np
import pytest

from decode_gemv_epilogue_gb300 import synth
from norm_util import assert_norms, norm_error
from oracle import gemv, quant, select

F16, Q8, Q4, Q4K = synth.F16, synth.Q8_0, synth.Q4_0, synth.Q4_K


def parts(n):
    """x as the sum of its n f16 parts, scaled to a power of two as the packed columns are."""
    def f(x):
        s = 2.0 ** (14 - np.floor(np.log2(np.abs(x).max(axis=-1, keepdims=True))))
        r, y = x * s, np.zeros_like(x)
        for _ in range(n):
            h = (r - y).astype(np.float16).astype(np.float64)
            y = y + h
        return y / s
    return f


def planted(raw, wt, E, x, M, K, ids, w, hold):
    """The experts' product with x and the gated values held as `hold` says, otherwise in 64 bits."""
    g, u, d = (select.quant_rows(r, E) for r in raw)
    y = np.zeros_like(x)
    for t in range(x.shape[0]):
        for e, c in zip(ids[t], w[t]):
            xt = hold(x[t])
            h = gemv.silu(quant.dequantize(g[e], wt, M, K) @ xt) * (quant.dequantize(u[e], wt, M, K) @ xt)
            y[t] += c * (quant.dequantize(d[e], wt, K, M) @ hold(h))
    return y


@pytest.mark.parametrize("wt", [F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("T, E, k, M, K", [(1, 8, 2, 256, 256), (5, 16, 8, 256, 768), (9, 4, 2, 512, 512)])
def test_lost_low_parts_are_seen(T, E, k, M, K, wt):
    dist = {Q8: (0.0005, 0.002), Q4: (0.005, 0.02), F16: 0.05}
    raw = [synth.weights(wt, E * r, c, seed=i, dist=dist.get(wt)) for i, (r, c) in enumerate(((M, K), (M, K), (K, M)))]
    rng = np.random.default_rng(9)
    x = rng.standard_normal((T, K)).astype(np.float32).astype(np.float64)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    w = rng.random((T, k))
    want, bound = select.experts(raw[0], raw[1], wt, raw[2], wt, E, x, M, K, ids, w)
    one, two = (planted(raw, wt, E, x, M, K, ids, w, parts(n)) for n in (1, 2))
    assert np.all(np.abs(one - want) <= bound)  # the elementwise bound does not see it
    with pytest.raises(AssertionError):
        assert_norms(one, want)
    assert norm_error(one, want) > 1e-4
    assert_norms(two, want, tol=5e-7)
