"""gemv_experts on the GPU against the fp64 oracle, every format, with the literal parity
tolerance of each product carried through the gated product and the down product."""

import numpy as np
import pytest

from decode_gemv_epilogue_gb300 import synth
from gpu_util import assert_within, dev_tensor
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
    def __init__(self, G, T, E, k, M, K, wt, wd, seed=0, shift=0):
        self.G, self.T, self.E, self.k, self.M, self.K, self.wt, self.wd = G, T, E, k, M, K, wt, wd
        dist = {Q8: (0.0005, 0.002), Q4: (0.005, 0.02), F16: 0.05}
        self.raw = [synth.weights(t, E * r, c, seed=seed + i, dist=dist.get(t))
                    for i, (t, r, c) in enumerate(((wt, M, K), (wt, M, K), (wd, K, M)))]
        rng = np.random.default_rng(seed + 9)
        self.x = rng.standard_normal((T, K)).astype(np.float32)
        self.ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if k <= E else \
            rng.integers(0, E, (T, k)).astype(np.int32)
        self.w = rng.random((T, k)).astype(np.float32)
        self.aux = rng.standard_normal((T, K)).astype(np.float32)
        self.dev = []
        for r in self.raw:  # `shift` bytes off a 256-byte boundary
            b = torch.zeros(r.size + 512, dtype=torch.uint8, device="cuda")
            b[shift:shift + r.size] = dev_tensor(r)
            self.dev.append(b[shift:])

    def run(self, aux="given", prepared=False, pdl=False, ids=None, x=None, w=None, norm=None):
        G, T, K = self.G, self.T, self.K
        ids = self.ids if ids is None else ids
        x = self.x if x is None else x
        n = G.experts_workspace(self.E, T, self.k, self.M, K)
        ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        dst = torch.full((T * K + 64,), -55.0, device="cuda")
        a = None
        if aux == "given":
            a = dev_tensor(self.aux)
        elif aux == "inplace":
            dst[:T * K] = dev_tensor(self.aux.reshape(-1))
            a = dst
        args = (self.dev[0], self.dev[1], self.wt, self.dev[2], self.wd, self.E, dev_tensor(x), self.M, K,
                dev_tensor(ids), dev_tensor(self.w if w is None else w), T, self.k, a, dst, ws)
        if prepared:
            graph = G.Graph([G.prepare_experts(*args, workspace_bytes=n, pdl=pdl)])
            graph.launch()
            if aux != "inplace":
                graph.launch()
        else:
            G.gemv_experts(*args, workspace_bytes=n, pdl=pdl, rms_norm_weight=None if norm is None else dev_tensor(norm),
                           rms_norm_eps=1e-6)
        torch.cuda.synchronize()
        assert torch.all(dst[T * K:] == -55.0) and torch.all(ws[n:] == 0xA5)
        return dst[:T * K].view(T, K).cpu().numpy()

    def want(self, aux=True, ids=None, x=None, w=None):
        return osel.experts(*self.raw[:2], self.wt, self.raw[2], self.wd, self.E, self.x if x is None else x, self.M,
                            self.K, self.ids if ids is None else ids, self.w if w is None else w,
                            self.aux if aux else None)

    def check(self, what=""):
        y, b = self.want()
        got = self.run()
        assert_within(got, y, b, what)
        assert np.array_equal(got.view(np.uint32), self.run(aux="inplace").view(np.uint32))
        assert np.array_equal(got.view(np.uint32), self.run(prepared=True, pdl=True).view(np.uint32))
        y, b = self.want(aux=False)
        assert_within(self.run(aux=None), y, b, what + " no aux")


SHAPES = [
    # T, E, k, M, K
    (1, 8, 2, 64, 256),
    (1, 4, 4, 96, 512),
    (2, 8, 3, 512, 256),
    (5, 16, 8, 256, 768),
    (9, 3, 2, 288, 1056),
    (33, 4, 2, 128, 512),
    (70, 2, 1, 64, 256),
    (256, 6, 2, 64, 288),
    (1, 1, 1, 32, 32),
]


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("T, E, k, M, K", SHAPES)
def test_formats(G, T, E, k, M, K, wt):
    if wt == Q4K:
        M, K = (M + 255) // 256 * 256, (K + 255) // 256 * 256
    Case(G, T, E, k, M, K, wt, wt).check()


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("T, E, k, M, K", [(40, 3, 1, 288, 256), (100, 4, 2, 512, 512), (256, 3, 2, 256, 768),
                                           (61, 5, 2, 96, 1056)])
def test_many_columns_per_expert(G, T, E, k, M, K, wt):
    if wt == Q4K:
        M, K = (M + 255) // 256 * 256, (K + 255) // 256 * 256
    Case(G, T, E, k, M, K, wt, wt, seed=15).check()


@pytest.mark.parametrize("wt, wd", [(Q4K, Q8), (Q4, F16), (F16, Q4), (Q8, Q4K), (F32, Q4), (Q4, F32)])
def test_mixed_formats(G, wt, wd):
    Case(G, 6, 5, 3, 256, 512, wt, wd, seed=20).check()
    Case(G, 60, 4, 2, 256, 512, wt, wd, seed=21).check()


@pytest.mark.parametrize("wt", [F32, F16])
@pytest.mark.parametrize("M, K", [(1, 1), (7, 33), (40, 100), (65, 31), (32, 48)])
def test_ragged_widths(G, M, K, wt):
    Case(G, 3, 4, 2, M, K, wt, wt, seed=30).check()


@pytest.mark.parametrize("wt", [F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("shift", [2, 8, 16])
def test_matrices_off_a_16_byte_boundary(G, wt, shift):
    Case(G, 3, 4, 2, 256, 256, wt, wt, seed=40, shift=shift).check()


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
def test_ids_without_an_expert(G, wt):
    c = Case(G, 6, 4, 3, 256, 256, wt, wt, seed=50)
    ids = c.ids.copy()
    ids[0] = -1
    ids[1, 1] = 4
    ids[2] = [-5, 2 ** 30, 1]
    ids[3] = 2  # one expert three times
    y, b = c.want(ids=ids)
    got = c.run(ids=ids)
    assert_within(got, y, b)
    assert np.array_equal(got[0], c.aux[0])
    none = np.full_like(ids, -1)
    assert np.array_equal(c.run(ids=none), c.aux)
    assert np.array_equal(c.run(ids=none, aux=None), np.zeros_like(c.aux))


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("T, k", [(1, 1), (1, 3), (1, 32), (2, 9), (5, 7), (7, 32), (8, 4), (31, 8), (40, 7), (256, 2)])
def test_every_choice_the_same_expert(G, T, k, wt):
    """A token may name an expert more than once, also more often than there are tokens."""
    c = Case(G, T, 3, k, 256, 256, wt, wt, seed=T + k)
    ids = np.full_like(c.ids, 2)
    y, b = c.want(ids=ids)
    assert_within(c.run(ids=ids), y, b)
    ids[T // 2, k // 2] = 0
    ids[0, 0] = -1
    y, b = c.want(ids=ids)
    assert_within(c.run(ids=ids), y, b)


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
def test_all_tokens_take_one_expert(G, wt):
    c = Case(G, 67, 3, 1, 256, 256, wt, wt, seed=60)
    ids = np.ones_like(c.ids)
    y, b = c.want(ids=ids)
    assert_within(c.run(ids=ids), y, b)


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
def test_scales_of_x(G, wt):
    """Columns of zeros, large and small values, and values over many magnitudes."""
    c = Case(G, 6, 4, 2, 256, 512, wt, wt, seed=70)
    x = c.x.copy()
    x[0] = 0.0
    x[1] *= 1e3
    x[2] *= 1e-12
    x[3] *= 10.0 ** np.random.default_rng(1).uniform(-6, 2, x.shape[1])
    x[4, 100:] = 0.0
    x[5] = 0.0
    x[5, 17] = 3.0
    y, b = c.want(x=x)
    assert_within(c.run(x=x), y, b)


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
def test_non_finite_values_stay_in_their_token(G, wt):
    c = Case(G, 5, 4, 2, 256, 256, wt, wt, seed=80)
    x = c.x.copy()
    x[1, 3] = np.nan
    x[3, 7] = np.inf
    got, ref = c.run(x=x), c.run()
    keep = [0, 2, 4]
    assert np.array_equal(got[keep].view(np.uint32), ref[keep].view(np.uint32))
    assert np.all(np.isnan(got[1])) and not np.any(np.isfinite(got[3]))
    w = c.w.copy()
    w[2, 1] = np.nan
    got = c.run(w=w)
    assert np.all(np.isnan(got[2]))
    assert np.array_equal(np.delete(got, 2, 0).view(np.uint32), np.delete(ref, 2, 0).view(np.uint32))


@pytest.mark.parametrize("wt, shift", [(F32, 0), (F16, 0), (Q8, 0), (Q4, 0), (Q4K, 0), (Q4, 2)])
@pytest.mark.parametrize("T", [1, 5, 70])
def test_rms_prologue(G, T, wt, shift):
    """x normalised as it is packed (or, off a 16-byte boundary, as it is read)."""
    c = Case(G, T, 6, 4, 256, 512, wt, wt, seed=100 + T, shift=shift)
    gam = (1.0 + 0.1 * synth.normal(c.K, seed=9)).astype(np.float32)
    xn = onorm.rms_norm(c.x, gam, 1e-6, c.K)
    y, b = c.want(x=xn)
    # the normalisation's own rounding: a tenth of the tolerance of each product (TOL_NORM_REL)
    assert_within(c.run(norm=gam), y, 1.1 * b)


def test_zero_ffn_width(G):
    c = Case(G, 2, 3, 2, 0, 64, F32, F32)
    assert np.array_equal(c.run(), c.aux)


def test_routed_step_as_one_graph(G):
    """Router logits, routing and the experts' product in one graph, on another stream."""
    c = Case(G, 8, 16, 4, 256, 512, Q4, Q4, seed=90)
    rw = synth.weights(F16, c.E, c.K, seed=91)
    x, rd = dev_tensor(c.x), dev_tensor(rw)
    logits = torch.empty(c.T, c.E, device="cuda")
    ids, w = torch.empty(c.T, c.k, dtype=torch.int32, device="cuda"), torch.empty(c.T, c.k, device="cuda")
    ws = torch.empty(G.experts_workspace(c.E, c.T, c.k, c.M, c.K), dtype=torch.uint8, device="cuda")
    dst = dev_tensor(c.aux)
    calls = [G.prepare(rd, F16, x, c.E, c.K, G.EPI_NONE, None, logits, ncols=c.T),
             G.prepare_route(logits, c.T, c.E, c.k, ids, w, pdl=True),
             G.prepare_experts(c.dev[0], c.dev[1], Q4, c.dev[2], Q4, c.E, x, c.M, c.K, ids, w, c.T, c.k, dst, dst, ws,
                               pdl=True)]
    graph = G.Graph(calls)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph.launch()
    s.synchronize()
    want_ids, want_w = osel.route(logits.cpu().numpy(), c.k)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    y, b = c.want(ids=want_ids, w=want_w)
    assert_within(dst.cpu().numpy(), y, b + 2e-6 * np.abs(y - c.aux))
