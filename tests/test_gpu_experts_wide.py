"""gemv_experts on the kernel of wide column groups, every block format: each case first asserts
that its shape takes that kernel."""

import numpy as np
import pytest

from decode_gemv_epilogue_gb300 import synth
from gpu_util import assert_within, dev_tensor
from oracle import gemv as ogemv
from oracle import norm as onorm
from oracle import select as osel
from test_select_plan import WIDE

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_experts import Case  # noqa: E402

Q8, Q4, Q4K = synth.Q8_0, synth.Q4_0, synth.Q4_K


@pytest.fixture(scope="module")
def G(lib):
    assert lib.device_status(reset=True) == 0
    yield lib
    assert lib.device_status() == 0, "a kernel reported a bounded-wait timeout"


def wide_case(G, wg, wd, T, E, k, M, K, seed):
    c = Case(G, T, E, k, M, K, wg, wd, seed=seed)
    ws = torch.empty(G.experts_workspace(E, T, k, M, K), dtype=torch.uint8, device="cuda")
    path, info = G.plan_experts(c.dev[0], c.dev[1], wg, c.dev[2], wd, E, dev_tensor(c.x), M, K, dev_tensor(c.ids),
                                dev_tensor(c.w), T, k, None, torch.empty(T * K, device="cuda"), ws)
    assert path == 4 and info["wide"] and info["wide_down"]
    return c


def uneven(T, k, E, counts, seed):
    """ids [T, k] in which expert e has counts[e] slots, in random places; the rest take none."""
    flat = np.concatenate([np.full(n, e) for e, n in enumerate(counts)])
    flat = np.concatenate([flat, np.full(T * k - flat.size, -1)])
    flat[-1:] = E  # an id past the experts, too
    return np.random.default_rng(seed).permutation(flat).astype(np.int32).reshape(T, k)


@pytest.mark.parametrize("case", WIDE)
def test_formats(G, case):
    wide_case(G, *case, seed=200).check()


@pytest.mark.parametrize("case", [WIDE[0], WIDE[3], WIDE[4], WIDE[5]])
@pytest.mark.parametrize("counts", [(1, 9, 16, 31), (7, 15, 32, 8), (256, 3, 0, 5), (0, 0, 0, 17), (12, 250, 243, 390)])
def test_uneven_experts(G, case, counts):
    """Groups of 1..7, 8, 9..15 and 16 columns, experts without any, slots without an expert."""
    c = wide_case(G, *case, seed=210)
    ids = uneven(c.T, c.k, c.E, counts, seed=211)
    y, b = c.want(ids=ids)
    got = c.run(ids=ids)
    assert_within(got, y, b)
    assert np.array_equal(got.view(np.uint32), c.run(ids=ids, aux="inplace").view(np.uint32))
    idle = np.all((ids < 0) | (ids >= c.E), axis=1)
    assert np.array_equal(got[idle], c.aux[idle])


@pytest.mark.parametrize("case", WIDE[:3])
def test_rms_prologue(G, case):
    c = wide_case(G, *case, seed=220)
    gam = (1.0 + 0.1 * synth.normal(c.K, seed=9)).astype(np.float32)
    y, b = c.want(x=onorm.rms_norm(c.x, gam, 1e-6, c.K))
    # the normalisation's own rounding: a tenth of the tolerance of each product (TOL_NORM_REL)
    assert_within(c.run(norm=gam), y, 1.1 * b)


@pytest.mark.parametrize("case", WIDE[:3])
def test_non_finite_values_stay_in_their_token(G, case):
    c = wide_case(G, *case, seed=230)
    x = c.x.copy()
    x[17, 3] = np.nan
    x[200, 70] = np.inf
    got, ref = c.run(x=x), c.run()
    assert np.array_equal(np.delete(got, (17, 200), 0).view(np.uint32), np.delete(ref, (17, 200), 0).view(np.uint32))
    assert np.all(np.isnan(got[17])) and not np.any(np.isfinite(got[200]))
    w = c.w.copy()
    w[99, 1] = np.nan
    got = c.run(w=w)
    assert np.all(np.isnan(got[99]))
    assert np.array_equal(np.delete(got, 99, 0).view(np.uint32), np.delete(ref, 99, 0).view(np.uint32))


def test_large_gated_values(G):
    """Gated values whose sum over a block is beyond float32 while each of them, and the product with
    Q4_K's mins, is not."""
    wg, wd, T, E, k, M, K = WIDE[-1]
    c = wide_case(G, wg, wd, T, E, k, M, K, seed=240)
    c.raw[1] = c.raw[0].copy()  # the same rows: silu(g) g > 0
    c.dev[1] = c.dev[0]
    x = c.x.astype(np.float64)
    W0 = ogemv.quant.dequantize(osel.quant_rows(c.raw[0], E)[0], wg, M, K)
    x[0] = np.linalg.solve(W0, np.full(M, 4.5e18))  # every gate of token 0 for expert 0
    x = x.astype(np.float32)
    h = ogemv.silu(W0 @ x[0]) * (W0 @ x[0])
    assert h.max() < 3e37 and h.reshape(-1, 32).sum(1).min() > 4e38
    ids, w = c.ids.copy(), c.w.copy()
    ids[0], w[0] = -1, 0.0
    ids[0, 0], w[0, 0] = 0, 0.25
    y, b = c.want(ids=ids, x=x, w=w)
    assert np.abs(y).max() < 1e38
    assert_within(c.run(ids=ids, x=x, w=w), y, b)
