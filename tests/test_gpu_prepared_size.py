"""What a prepared call keeps on the host: its own launches, not room for the longest call's."""

import pytest

from decode_gemv_epilogue_gb300 import synth
from gpu_util import dev_tensor

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def resident():
    with open("/proc/self/statm") as f:
        return int(f.read().split()[1]) * 4096


def test_handles_are_small(lib):
    W, x = dev_tensor(synth.weights(synth.Q4_0, 64, 256, seed=1)), torch.zeros(256, device="cuda")
    y, ids, w = torch.zeros(64, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda"), torch.zeros(8, device="cuda")

    def make(n):
        return [lib.prepare(W, synth.Q4_0, x, 64, 256, 0, None, y) for _ in range(n)] + \
            [lib.prepare_route(x, 1, 64, 8, ids, w) for _ in range(n)]

    first = make(10)
    before = resident()
    calls = make(2000)
    grown = resident() - before
    assert grown <= 4000 * 4096, "%.0f bytes a handle" % (grown / 4000)
    lib.launch_prepared(calls[:2] + calls[-2:])
    torch.cuda.synchronize()
    assert lib.device_status() == 0 and len(first) == 20
