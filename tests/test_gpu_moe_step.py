"""The mixture-of-experts step: adapters, router, routing and experts in one graph, each stage
against the fp64 oracle on the stage's own inputs."""

import numpy as np
import pytest

from decode_gemv_epilogue_gb300 import synth
from gpu_util import TOL_NORM_REL, assert_within
from oracle import gemv as ogemv
from oracle import norm as onorm
from oracle import select as osel

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.mark.parametrize("T, d, ffn, E, k, wt", [(1, 512, 256, 8, 2, synth.Q4_0), (5, 256, 96, 6, 3, synth.Q8_0),
                                                 (20, 512, 256, 4, 2, synth.Q4_K)])
def test_step(lib, T, d, ffn, E, k, wt):
    from decode_gemv_epilogue_gb300.moe_step import MoeStep
    s = MoeStep(T, d, ffn, E, k, n_adapters=3, rank=8, wtype=wt, seed=T)
    x = synth.normal(T * d, seed=99).astype(np.float32).reshape(T, d)
    s.x.copy_(torch.from_numpy(x))
    s.adapters.copy_(torch.arange(T, dtype=torch.int32) % 4 - 1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s.launch(stream=side)
    s.launch(stream=side)  # again over the same buffers: the same result
    side.synchronize()
    g = {n: getattr(s, n).cpu().numpy() for n in ("h", "logits", "ids", "weights", "y", "adapters")}
    h = s.host
    A, B = h["A"].reshape(3, 8, d), h["B"].reshape(3, d, 8)
    want, b = osel.lora(h["wo"], wt, x, d, d, ogemv.EPI_ADD, x, A, B, g["adapters"], h["scales"])
    assert_within(g["h"], want, b, "projection")
    n = onorm.rms_norm(g["h"], h["gamma"], s.eps, d)
    want = ogemv.gemv(h["router"], synth.F16, n, E, d)
    b = (2e-5 + TOL_NORM_REL) * ogemv.abs_dot(h["router"], synth.F16, n, E, d) + 1e-6
    assert_within(g["logits"], want, b, "logits")
    ids, w = osel.route(g["logits"], k)
    assert np.array_equal(g["ids"], ids)
    assert np.all(np.abs(g["weights"] - w) <= 1e-5 * w)
    # the normalisation's own rounding: a tenth of the tolerance of each product (TOL_NORM_REL)
    want, b = osel.experts(h["gate"], h["up"], wt, h["down"], wt, E, n, ffn, d, g["ids"], g["weights"], g["h"])
    assert_within(g["y"], want, 1.1 * b, "experts")
    assert lib.device_status() == 0
