"""Which kernels gemv_experts and gemv_lora choose (host only): the queries themselves, and the
shapes on which the GPU tests rely to reach each kernel.  Pointers are fake device addresses."""

import pytest

from decode_gemv_epilogue_gb300 import synth

F32, F16, Q8, Q4, Q4K = synth.F32, synth.F16, synth.Q8_0, synth.Q4_0, synth.Q4_K
BASE = [i << 40 for i in range(1, 12)]

# (gate and up, down, T, E, k, M, K) whose column groups are 16 wide: tests/test_gpu_experts_wide.py
WIDE = [
    (Q8, Q8, 256, 4, 4, 256, 512),
    (Q4, Q4, 256, 4, 4, 512, 512),
    (Q4K, Q4K, 256, 4, 4, 512, 512),
    (Q4, Q4, 256, 4, 4, 256, 768),
    (Q4K, Q4K, 256, 4, 4, 256, 768),
    (Q4K, Q8, 256, 4, 4, 512, 256),
    (Q8, Q4, 200, 4, 4, 256, 768),
    (Q4, Q4K, 256, 8, 8, 256, 256),
]


def experts(lib, wg, wd, T, E, k, M, K, shift=0, **kw):
    g, u, d, x, i, w, dst, ws = BASE[:8]
    return lib.plan_experts(g + shift, u, wg, d, wd, E, x, M, K, i, w, T, k, None, dst, ws, workspace_bytes=1 << 39, **kw)


def lora(lib, wt, N, M, K, n=4, r=16, epi=0, **kw):
    W, x, dst, A, B, i, s, ws = BASE[:8]
    return lib.plan_lora(W, wt, x, M, K, epi, None, dst, A, B, F16, n, r, i, s, ws, workspace_bytes=1 << 39, ncols=N, **kw)


@pytest.mark.parametrize("case", WIDE)
def test_wide_groups(lib, case):
    assert experts(lib, *case) == (4, dict(cols=16, wide=True, wide_down=True))


@pytest.mark.parametrize("wt, T, E, k, cols", [(Q4, 1, 8, 2, 1), (Q8, 5, 8, 2, 5), (Q4K, 9, 8, 2, 8), (F16, 9, 8, 2, 8),
                                               (F16, 60, 8, 1, 16), (F32, 60, 8, 1, 16), (F16, 256, 8, 2, 24)])
def test_narrow_groups(lib, wt, T, E, k, cols):
    assert experts(lib, wt, wt, T, E, k, 512, 512) == (4, dict(cols=cols, wide=False, wide_down=False))


def test_experts_other_answers(lib):
    assert experts(lib, Q4, Q4, 4, 8, 2, 256, 256, shift=8)[0] == 2  # off a 16-byte boundary
    assert experts(lib, F16, F16, 4, 8, 2, 250, 256)[0] == 2
    assert experts(lib, F16, F16, 4, 8, 2, 0, 256)[0] == 2
    assert experts(lib, Q4, Q4, 4, 8, 2, 256, 256)[0] == 4
    assert experts(lib, Q4, Q4, 4, 8, 2, 256, 256, tensor_cores=False)[0] == 2
    assert experts(lib, Q4, Q4, 0, 8, 2, 256, 256)[0] == 0
    assert experts(lib, Q4, Q4, 257, 8, 2, 256, 256)[0] == lib.ERR_UNSUPPORTED
    assert experts(lib, Q4, Q4, 4, 8, 9, 256, 0)[0] == 0
    assert lib.raw.gf_plan_experts(None, BASE[0], 1, None, BASE[1], None) == lib.ERR_INVALID


def test_lora_answers(lib):
    assert lora(lib, Q4, 64, 14336, 4096) == (4, dict(cols=16, wide=True))
    assert lora(lib, Q4, 64, 600, 1024) == (4, dict(cols=8, wide=False))
    assert lora(lib, F16, 64, 600, 1056) == (4, dict(cols=16, wide=False))
    assert lora(lib, Q4, 1, 600, 1024)[0] == 1
    assert lora(lib, F16, 8, 4096, 4096)[0] == 3
    assert lora(lib, Q4, 64, 600, 1024, tensor_cores=False)[0] == 1
    assert lora(lib, Q4, 64, 600, 1024, n=0)[0] == 1
    assert lora(lib, F32, 4, 600, 33)[0] == 2
    assert lora(lib, Q4, 64, 0, 1024)[0] == 0
    assert lora(lib, Q4, 64, 600, 1024, r=257)[0] == lib.ERR_UNSUPPORTED
    assert lib.raw.gf_plan_lora(BASE[0], Q4, BASE[1], 8, 32, 0, None, BASE[2], None, None, None) == lib.ERR_INVALID


@pytest.mark.parametrize("M, path", [(1 << 30, 4), ((1 << 30) + 64, 1), ((1 << 31) - 8, 1)])
def test_lora_rows_near_the_end_of_32_bits(lib, M, path):
    """The tiled kernels count rows, rounded up to a tile, in 32 bits."""
    assert lora(lib, Q4, 17, M, 256)[0] == path
