"""gemv_experts and gemv_lora on the GPU: every output vector against the fp64 oracle by its norm,
over the formats and the kernels."""

import numpy as np
import pytest

from decode_gemv_epilogue_gb300 import synth
from gpu_util import dev_tensor
from norm_util import assert_norms

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import test_gpu_experts  # noqa: E402
import test_gpu_lora  # noqa: E402

F32, F16, Q8, Q4, Q4K = synth.F32, synth.F16, synth.Q8_0, synth.Q4_0, synth.Q4_K
ALL = [F32, F16, Q8, Q4, Q4K]


@pytest.fixture(scope="module")
def G(lib):
    assert lib.device_status(reset=True) == 0
    yield lib
    assert lib.device_status() == 0, "a kernel reported a bounded-wait timeout"


# (T, E, k, M, K, bytes off a 16-byte boundary, path, columns of a group: block formats, F16 and F32)
KERNELS = {
    "one": (1, 8, 2, 256, 512, 0, 4, 1, 1),
    "few": (4, 8, 3, 256, 768, 0, 4, 4, 4),
    "five": (5, 16, 8, 256, 768, 0, 4, 5, 5),
    "tile": (40, 16, 4, 512, 512, 0, 4, 8, 16),
    "many": (256, 4, 4, 512, 512, 0, 4, 16, 24),
    "generic": (5, 6, 2, 256, 512, 4, 2, 0, 0),
}


@pytest.mark.parametrize("wt", ALL)
@pytest.mark.parametrize("kind", list(KERNELS))
def test_experts(G, wt, kind):
    T, E, k, M, K, shift, path, block, plain = KERNELS[kind]
    c = test_gpu_experts.Case(G, T, E, k, M, K, wt, wt, seed=500 + T, shift=shift)
    ws = torch.empty(G.experts_workspace(E, T, k, M, K), dtype=torch.uint8, device="cuda")
    got, info = G.plan_experts(c.dev[0], c.dev[1], wt, c.dev[2], wt, E, dev_tensor(c.x), M, K, dev_tensor(c.ids),
                               dev_tensor(c.w), T, k, None, torch.empty(T * K, device="cuda"), ws)
    assert got == path and info["cols"] == (plain if wt in (F32, F16) else block)
    print("off by %.3g" % assert_norms(c.run(aux=None), c.want(aux=False)[0], kind))


@pytest.mark.parametrize("wg, wd", [(Q4K, Q8), (Q8, Q4), (Q4, Q4K), (F16, Q4), (Q4, F16)])
@pytest.mark.parametrize("T", [3, 256])
def test_experts_mixed(G, T, wg, wd):
    c = test_gpu_experts.Case(G, T, 4, 4, 256, 768, wg, wd, seed=520 + T)
    print("off by %.3g" % assert_norms(c.run(aux=None), c.want(aux=False)[0]))


@pytest.mark.parametrize("wt", ALL)
@pytest.mark.parametrize("N, M, K", [(1, 300, 512), (3, 16384, 1024), (8, 8200, 1024), (40, 300, 512), (250, 4500, 512)])
def test_lora(G, N, M, K, wt):
    c = test_gpu_lora.Case(G, N, M, K, wt, 3, 8, F16, seed=540 + N)
    c.ids[:] = np.arange(N) % 4 - 1
    print("off by %.3g" % assert_norms(c.run(0), c.want(0)[0]))


@pytest.mark.parametrize("wt", ALL)
def test_experts_without_tensor_cores(G, wt):
    """The generic kernels where the tiled ones would take the call: 32 bits throughout."""
    T, E, k, M, K = 9, 4, 2, 256, 512
    c = test_gpu_experts.Case(G, T, E, k, M, K, wt, wt, seed=560)
    ws = torch.empty(G.experts_workspace(E, T, k, M, K), dtype=torch.uint8, device="cuda")
    dst = torch.empty(T, K, device="cuda")
    args = (c.dev[0], c.dev[1], wt, c.dev[2], wt, E, dev_tensor(c.x), M, K, dev_tensor(c.ids), dev_tensor(c.w), T, k, None,
            dst, ws)
    assert G.plan_experts(*args)[0] == 4 and G.plan_experts(*args, tensor_cores=False)[0] == 2
    G.gemv_experts(*args, tensor_cores=False)
    torch.cuda.synchronize()
    got = dst.cpu().numpy()
    assert_norms(got, c.want(aux=False)[0], tol=1e-6)
    graph = G.Graph([G.prepare_experts(*args, tensor_cores=False)])
    dst.zero_()
    graph.launch()
    torch.cuda.synchronize()
    assert np.array_equal(got.view(np.uint32), dst.cpu().numpy().view(np.uint32))
