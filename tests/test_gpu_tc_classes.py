"""Infinities and NaN in x through the tensor-core kernel of F16 batches, alone and beside adapters:
the oracle's NaN and infinities, whatever the batch."""

import numpy as np
import pytest

from decode_gemv_epilogue_gb300 import synth
from gpu_util import assert_within, dev_tensor, gemv_bound
from oracle import gemv as ogemv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import test_gpu_lora  # noqa: E402
from test_gpu_select_range import assert_classes  # noqa: E402

F16 = synth.F16


@pytest.fixture(scope="module")
def G(lib):
    assert lib.device_status(reset=True) == 0
    yield lib
    assert lib.device_status() == 0, "a kernel reported a bounded-wait timeout"


def with_bad(X):
    """Column 0 with +inf, 1 with -inf and a NaN elsewhere, 2 with +inf beside values of 1e30."""
    X = X.copy()
    X[0, 37] = np.inf
    X[1, 70] = -np.inf if X.shape[0] > 3 else np.nan
    X[2, 5], X[2, 100:300] = np.inf, 1e30
    if X.shape[0] > 4:
        X[3, 9] = np.nan
        X[4, 9], X[4, 400] = np.inf, -np.inf
    return X


@pytest.mark.parametrize("M, K, ncols", [(300, 512, 3), (4096, 1024, 8), (520, 5120, 16), (20000, 512, 5), (700, 512, 40)])
@pytest.mark.parametrize("epi", [ogemv.EPI_NONE, ogemv.EPI_SIGMOID, ogemv.EPI_ADD])
def test_plain_batches(G, M, K, ncols, epi):
    raw = synth.weights(F16, M, K, seed=700 + ncols)
    w = raw.view(np.float16).reshape(M, K)
    w[::7, 37] = 0  # 0 * inf: NaN
    X = with_bad(synth.normal(ncols * K, seed=701).reshape(ncols, K))
    aux = synth.normal(ncols * M, seed=702).reshape(ncols, M)
    Wd, xd = dev_tensor(raw), dev_tensor(X)
    dst = dev_tensor(aux.copy()) if epi == ogemv.EPI_ADD else torch.empty(ncols, M, device="cuda")
    a = dst if epi == ogemv.EPI_ADD else None
    assert G.plan(Wd, F16, xd, M, K, epi, a, dst, ncols=ncols)[0] == 3
    G.gemv_fused_ex(Wd, F16, xd, M, K, epi, a, dst, ncols=ncols)
    torch.cuda.synchronize()
    got = dst.cpu().numpy()
    with np.errstate(invalid="ignore", over="ignore"):
        want = ogemv.gemv(raw, F16, X, M, K, epi, aux)
    assert_classes(got, want)
    fin = np.isfinite(X).all(axis=1)
    assert_within(got[fin], want[fin], gemv_bound(raw, F16, X[fin], M, K))


@pytest.mark.parametrize("N", [3, 8, 40])
def test_beside_adapters(G, N):
    c = test_gpu_lora.Case(G, N, 300, 512, F16, 3, 8, F16, seed=710)
    c.ids[:5] = -1
    x = with_bad(c.x)
    ws = torch.empty(G.lora_workspace(N, 300, 512, c.r, c.n), dtype=torch.uint8, device="cuda")
    assert G.plan_lora(c.Wd, F16, dev_tensor(x), 300, 512, 1, None, torch.empty(N * 300, device="cuda"), c.Ad, c.Bd, F16,
                       c.n, c.r, dev_tensor(c.ids), None, ws, ncols=N)[0] == 3
    for epi in (0, 1):
        got = c.run(epi, x=x)
        with np.errstate(invalid="ignore", over="ignore"):
            want, _ = c.want(epi, x=x)
        assert_classes(got, want)
