"""Guard bands around every operand of routing, the experts' product and the adapters: 4 KiB of a
known byte before and behind each of them, untouched after calls on ragged shapes through every
kernel; the outputs are checked too, so that no band stays clean because nothing was written."""

import numpy as np
import pytest

from decode_gemv_epilogue_gb300 import synth
from gpu_util import assert_within, dev_tensor
from oracle import gemv as ogemv
from oracle import select as osel

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import test_gpu_experts  # noqa: E402
import test_gpu_lora  # noqa: E402
import test_gpu_redzone as rz  # noqa: E402

F32, F16, Q8, Q4, Q4K = synth.F32, synth.F16, synth.Q8_0, synth.Q4_0, synth.Q4_K


@pytest.fixture(scope="module")
def G(lib):
    assert lib.device_status(reset=True) == 0
    yield lib
    assert lib.device_status() == 0, "a kernel reported a bounded-wait timeout"


class Guarded:
    """A device tensor between two bands.  `at`: bytes it lies off a 4 KiB boundary."""

    def __init__(self, arr=None, n=None, dtype=torch.float32, at=0):
        t = torch.from_numpy(np.ascontiguousarray(arr).reshape(-1)) if arr is not None else torch.zeros(n, dtype=dtype)
        self.nbytes = t.numel() * t.element_size()
        self.lo = rz.GUARD + at
        raw = torch.full((self.lo + self.nbytes + rz.GUARD + 4096,), rz.PAT, dtype=torch.uint8, device="cuda")
        base = -raw.data_ptr() % 4096
        self.buf = raw[base:base + self.lo + self.nbytes + rz.GUARD]
        self.t = self.buf[self.lo:self.lo + self.nbytes].view(t.dtype)
        self.t.copy_(t)

    def intact(self):
        lo, hi = self.buf[:self.lo], self.buf[self.lo + self.nbytes:]
        return bool(torch.all(lo == rz.PAT)) and bool(torch.all(hi == rz.PAT))


@pytest.mark.parametrize("T, E, k, groups, ld", [(1, 1, 1, 1, 0), (7, 60, 4, 1, 61), (61, 256, 8, 8, 0), (300, 33, 32, 1, 40),
                                                 (5, 1024, 3, 32, 1030)])
def test_route(G, T, E, k, groups, ld):
    rng = np.random.default_rng(T + E)
    logits = rng.standard_normal((T, ld or E)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    L, B = Guarded(logits.reshape(-1)[:(T - 1) * (ld or E) + E], at=4), Guarded(bias, at=8)
    I, W = Guarded(n=T * k, dtype=torch.int32, at=4), Guarded(n=T * k, at=12)
    keep = max(1, groups // 2)
    for b in (None, B):
        G.route(L.t, T, E, k, I.t, W.t, score=G.SCORE_SIGMOID, bias=None if b is None else b.t, n_group=groups,
                topk_group=keep, ld=ld)
        rz.check_all(L, B, I, W)
        ids, w = osel.route(logits[:, :E], k, score="sigmoid", bias=None if b is None else bias, n_group=groups,
                            topk_group=keep)
        assert np.array_equal(I.t.view(T, k).cpu().numpy(), ids)
        assert np.all(np.abs(W.t.view(T, k).cpu().numpy() - w) <= 1e-5 * np.abs(w) + 1e-30)


# T, E, k, M, K, bytes off a boundary: one column, few, a tile, the wide kernel, the generic ones
EXPERTS = [(1, 4, 3, 32, 32, 0), (3, 5, 2, 96, 160, 0), (9, 3, 2, 288, 1056, 0), (33, 4, 2, 64, 96, 0),
           (256, 8, 8, 256, 256, 0), (5, 4, 2, 64, 96, 2)]


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("T, E, k, M, K, at", EXPERTS)
def test_experts(G, T, E, k, M, K, at, wt):
    if wt == Q4K:
        M, K = (M + 255) // 256 * 256, (K + 255) // 256 * 256
    if wt == F32:
        at *= 2
    c = test_gpu_experts.Case(G, T, E, k, M, K, wt, wt, seed=600 + T)
    ids = c.ids.copy()
    ids.reshape(-1)[::5] = -1
    gam = (1.0 + 0.1 * synth.normal(K, seed=601)).astype(np.float32)
    n = G.experts_workspace(E, T, k, M, K)
    ops = [Guarded(r, at=at) for r in c.raw] + [Guarded(c.x, at=4 if at else 0), Guarded(ids, at=4), Guarded(c.w, at=8),
                                                Guarded(c.aux, at=4), Guarded(gam, at=4 if at else 0),
                                                Guarded(n=n, dtype=torch.uint8), Guarded(n=T * K, at=12)]
    g, u, d, x, i, w, aux, gm, ws, dst = ops
    G.gemv_experts(g.t, u.t, wt, d.t, wt, E, x.t, M, K, i.t, w.t, T, k, aux.t, dst.t, ws.t)
    rz.check_all(*ops)
    want, b = c.want(ids=ids)
    assert_within(dst.t.view(T, K).cpu().numpy(), want, b)
    G.gemv_experts(g.t, u.t, wt, d.t, wt, E, x.t, M, K, i.t, w.t, T, k, None, dst.t, ws.t, rms_norm_weight=gm.t,
                   rms_norm_eps=1e-6)
    x.t[0] = float("inf")  # and the way of columns that are not packed
    G.gemv_experts(g.t, u.t, wt, d.t, wt, E, x.t, M, K, i.t, w.t, T, k, aux.t, aux.t, ws.t)
    rz.check_all(*ops)


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("N, M, K, r, at", [(1, 33, 256, 5, 2), (3, 10007, 4608, 16, 0), (9, 302, 1056, 8, 0), (20, 131, 1056, 24, 0),
                                            (70, 1001, 512, 64, 0), (250, 4499, 256, 16, 0)])
def test_lora(G, N, M, K, r, at, wt):
    if wt == Q4K:
        K = (K + 255) // 256 * 256
    c = test_gpu_lora.Case(G, N, M, K, wt, 4, r, F16, seed=610 + N)
    n = G.lora_workspace(N, M, K, r, 4)
    ops = [Guarded(c.raw), Guarded(c.x), Guarded(c.A, at=at), Guarded(c.B, at=at), Guarded(c.ids, at=4), Guarded(c.scales, at=4),
           Guarded(c.aux, at=4), Guarded(n=n, dtype=torch.uint8), Guarded(n=N * M, at=4)]
    W, x, A, B, i, s, aux, ws, dst = ops
    for epi in (ogemv.EPI_SILU, ogemv.EPI_SILU_MUL):
        G.gemv_lora(W.t, wt, x.t, M, K, epi, aux.t if epi == ogemv.EPI_SILU_MUL else None, dst.t, A.t, B.t, F16, 4, r, i.t,
                    s.t, ws.t, ncols=N)
        rz.check_all(*ops)
        want, b = c.want(epi)
        assert_within(dst.t.view(N, M).cpu().numpy(), want, b)
    x.t[K // 2] = float("inf")
    G.gemv_lora(W.t, wt, x.t, M, K, ogemv.EPI_ADD, aux.t, aux.t, A.t, B.t, F16, 4, r, i.t, s.t, ws.t, ncols=N)
    rz.check_all(*ops)
