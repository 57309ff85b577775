"""gemv_lora on the GPU against the fp64 oracle: every format and tail, adapters of either
type, columns without one, batches over every kernel of the shared product."""

import numpy as np
import pytest

from decode_gemv_epilogue_gb300 import synth
from gpu_util import TOL_NORM_REL, assert_within, dev_tensor
from oracle import fwht as ofwht
from oracle import gemv as ogemv
from oracle import norm as onorm
from oracle import select as osel

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

F32, F16, Q8, Q4, Q4K = synth.F32, synth.F16, synth.Q8_0, synth.Q4_0, synth.Q4_K


@pytest.fixture(scope="module")
def G(lib):
    assert lib.device_status(reset=True) == 0
    yield lib
    assert lib.device_status() == 0, "a kernel reported a bounded-wait timeout"


class Case:
    def __init__(self, G, N, M, K, wt, n, r, at, seed=0, shift=0):
        self.G, self.N, self.M, self.K, self.wt, self.n, self.r, self.at = G, N, M, K, wt, n, r, at
        rng = np.random.default_rng(seed)
        self.raw = synth.weights(wt, M, K, seed=seed)
        t = np.float16 if at == F16 else np.float32
        self.A = (rng.standard_normal((n, r, K)) * K ** -0.5).astype(t)
        self.B = (rng.standard_normal((n, M, r)) * r ** -0.5).astype(t)
        self.scales = (0.5 + rng.random(n)).astype(np.float32)
        self.ids = rng.integers(0, n, N).astype(np.int32)
        if N > 1:
            self.ids[rng.integers(0, N)] = -1
        if N > 3:
            self.ids[0], self.ids[3] = n, 2 ** 30
        self.x = rng.standard_normal((N, K)).astype(np.float32)
        self.aux = rng.standard_normal((N, M)).astype(np.float32)
        self.Wd = dev_tensor(self.raw)
        self.Ad, self.Bd = (torch.cat([torch.zeros(shift, dtype=b.dtype, device="cuda"), b.reshape(-1)])[shift:]
                            for b in (dev_tensor(self.A), dev_tensor(self.B)))

    def run(self, epi, inplace=False, prepared=False, scales=True, ids=None, x=None, **opts):
        G, N, M = self.G, self.N, self.M
        n = G.lora_workspace(N, M, self.K, self.r, self.n)
        ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        dst = torch.full((N * M + 64,), -55.0, device="cuda")
        aux = None
        if epi in ogemv.NEEDS_AUX:
            aux = dev_tensor(self.aux)
            if inplace:
                dst[:N * M] = aux.reshape(-1)
                aux = dst
        args = (self.Wd, self.wt, dev_tensor(self.x if x is None else x), M, self.K, epi, aux, dst, self.Ad, self.Bd,
                self.at, self.n, self.r, dev_tensor(self.ids if ids is None else ids),
                dev_tensor(self.scales) if scales else None, ws)
        if prepared:
            graph = G.Graph([G.prepare_lora(*args, workspace_bytes=n, ncols=N, **opts)])
            graph.launch()
            if not inplace:
                graph.launch()
        else:
            G.gemv_lora(*args, workspace_bytes=n, ncols=N, **opts)
        torch.cuda.synchronize()
        assert torch.all(dst[N * M:] == -55.0) and torch.all(ws[n:] == 0xA5)
        return dst[:N * M].view(N, M).cpu().numpy()

    def want(self, epi, scales=True, ids=None, x=None):
        return osel.lora(self.raw, self.wt, self.x if x is None else x, self.M, self.K, epi,
                         self.aux if epi in ogemv.NEEDS_AUX else None, self.A, self.B, self.ids if ids is None else ids,
                         self.scales if scales else None)

    def check(self, epi):
        y, b = self.want(epi)
        got = self.run(epi)
        assert_within(got, y, b, "epilogue %d" % epi)
        assert np.array_equal(got.view(np.uint32), self.run(epi, prepared=True, pdl=True).view(np.uint32))
        if epi in ogemv.NEEDS_AUX:
            assert np.array_equal(got.view(np.uint32), self.run(epi, inplace=True).view(np.uint32))


@pytest.mark.parametrize("epi", range(5))
@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("N", [1, 3, 8, 19])
def test_formats_and_tails(G, N, wt, epi):
    Case(G, N, 200, 512, wt, 4, 16, F16, seed=N).check(epi)


@pytest.mark.parametrize("at", [F16, F32])
@pytest.mark.parametrize("r", [1, 3, 8, 24, 64, 100, 256])
def test_ranks(G, r, at):
    Case(G, 5, 136, 768, Q8, 3, r, at, seed=r).check(4)


@pytest.mark.parametrize("at", [F16, F32])
@pytest.mark.parametrize("M, K", [(1, 1), (5, 33), (300, 100), (257, 2056), (64, 4100)])
def test_ragged_shapes(G, M, K, at):
    Case(G, 4, M, K, F32, 3, 12, at, seed=M).check(2)


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4])
@pytest.mark.parametrize("N, M, K", [(60, 700, 1056), (2, 8, 32), (3, 71, 96), (9, 302, 3648), (20, 131, 1056), (33, 100, 1984)])
def test_rows_of_no_whole_16_byte_words(G, N, M, K, wt):
    """Block-format batches whose rows a tensor map reaches only several at a time, and rows
    left over at the end."""
    c = Case(G, N, M, K, wt, 3, 8, F16, seed=M + K)
    c.check(1)
    c.check(4)


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("N, M, K", [(2, 8, 256), (9, 33, 512), (16, 1000, 768), (17, 513, 256), (64, 600, 1024),
                                     (70, 1000, 1024), (3, 10000, 4608), (8, 4100, 4096)])
def test_batches(G, N, M, K, wt):
    c = Case(G, N, M, K, wt, 5, 16, F16, seed=N)
    c.check(2)
    c.check(3)


@pytest.mark.parametrize("wt", [Q8, Q4, Q4K])
@pytest.mark.parametrize("N, M, K", [(125, 4009, 256), (64, 13101, 256), (57, 18002, 512), (250, 4500, 768)])
def test_wide_batches_of_many_rows(G, N, M, K, wt):
    """Enough rows and columns for the kernel of wide column groups, its items of 8, 12 and 16
    warps' rows, the last item ragged."""
    Case(G, N, M, K, wt, 9, 16, F16, seed=M).check(3)


@pytest.mark.parametrize("at", [F16, F32])
@pytest.mark.parametrize("shift", [1, 4])
def test_adapters_off_a_16_byte_boundary(G, at, shift):
    Case(G, 3, 100, 512, Q4, 2, 16, at, seed=3, shift=shift).check(0)


@pytest.mark.parametrize("wt", [F16, Q4])
def test_widest_batch(G, wt):
    Case(G, 256, 96, 512, wt, 7, 32, F16, seed=4).check(3)


def test_one_adapter_for_all_and_none_at_all(G):
    c = Case(G, 33, 300, 512, Q4, 3, 16, F16, seed=5)
    ids = np.ones_like(c.ids)
    y, b = c.want(0, ids=ids)
    assert_within(c.run(0, ids=ids), y, b)
    ids[:] = -1
    y, b = c.want(2, ids=ids)
    assert_within(c.run(2, ids=ids), y, b)


def test_without_scales(G):
    c = Case(G, 3, 64, 256, Q4, 2, 8, F16, seed=6)
    y, b = c.want(0, scales=False)
    assert_within(c.run(0, scales=False), y, b)


def test_split_rows(G):
    """Few rows and a long K: the shared product splits K over clusters."""
    c = Case(G, 1, 24, 32768, Q4, 2, 16, F16, seed=7)
    c.check(1)


@pytest.mark.parametrize("N, M, wt", [(1, 128, Q4), (3, 128, Q4), (3, 130, Q8), (18, 64, Q4K), (4, 96, F16)])
def test_rms_prologue(G, N, M, wt):
    c = Case(G, N, M, 1024, wt, 3, 16, F16, seed=8)
    if wt == Q8:  # rows a tensor map reaches two at a time, two rows left over
        c = Case(G, N, M, 1120, wt, 3, 16, F16, seed=8)
    gam, eps = (1.0 + 0.1 * synth.normal(c.K, seed=9)).astype(np.float32), 1e-6
    xn = onorm.rms_norm(c.x, gam, eps, c.K)
    y, b = c.want(4, x=xn)
    extra = TOL_NORM_REL * (ogemv.abs_dot(c.raw, c.wt, xn, c.M, c.K))
    for q, a in enumerate(c.ids):
        if 0 <= a < c.n:
            extra[q] += TOL_NORM_REL * c.scales[a] * (np.abs(c.B[a].astype(float)) @
                                                     (np.abs(c.A[a].astype(float)) @ np.abs(xn[q])))
    got = c.run(4, rms_norm_weight=dev_tensor(gam), rms_norm_eps=eps)
    assert_within(got, y, b + extra)


def test_fwht_prologue(G):
    c = Case(G, 4, 128, 1024, F16, 3, 16, F16, seed=10)
    s = synth.rademacher(256, seed=11)
    xp = np.stack([ofwht.fwht_signed(c.x[q], s, 256) for q in range(c.N)])
    e = np.stack([ofwht.fwht_abs_scale(c.x[q], 256) * 2e-5 + 1e-6 for q in range(c.N)])
    y, b = c.want(0, x=xp)
    b = b + ogemv.abs_w_dot(c.raw, c.wt, e, c.M, c.K)
    for q, a in enumerate(c.ids):
        if 0 <= a < c.n:
            b[q] += c.scales[a] * (np.abs(c.B[a].astype(float)) @ (np.abs(c.A[a].astype(float)) @ e[q]))
    ws = torch.empty(c.N * c.K, device="cuda")
    got = c.run(0, fwht_signs=dev_tensor(s), fwht_block=256, nsigns=256, fwht_workspace=ws)
    assert_within(got, y, b)


def test_non_finite_values_stay_in_their_column(G):
    c = Case(G, 5, 96, 512, F32, 2, 8, F16, seed=12)
    c.ids[:] = [0, 1, 0, 1, 0]
    x = c.x.copy()
    x[1, 3] = np.nan
    x[3, 5] = np.inf
    got, ref = c.run(0, x=x), c.run(0)
    assert np.array_equal(got[[0, 2, 4]].view(np.uint32), ref[[0, 2, 4]].view(np.uint32))
    assert np.all(np.isnan(got[1])) and not np.any(np.isfinite(got[3]))


def test_no_adapters_loaded(G):
    c = Case(G, 2, 64, 256, Q4, 1, 8, F16, seed=13)
    c.n = 0
    ref = torch.empty(2 * 64, device="cuda")
    G.gemv_fused_ex(c.Wd, Q4, dev_tensor(c.x), 64, 256, 0, None, ref, ncols=2)
    torch.cuda.synchronize()
    assert np.array_equal(c.run(0), ref.view(2, 64).cpu().numpy())


def test_other_stream(G):
    c = Case(G, 4, 128, 512, Q4, 3, 16, F16, seed=14)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = c.run(0)
    y, b = c.want(0)
    assert_within(got, y, b)
