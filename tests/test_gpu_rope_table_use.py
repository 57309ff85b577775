"""A rotation table of another n_rot than a call's own: nothing of it behind its header is read, nothing is written,
and gf_device_status says so.  (Every table here lies at the start of a buffer that is long enough for any.)"""

import numpy as np
import pytest

import attend_util as au
from gpu_util import dev_tensor

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(scope="module")
def G(lib):
    assert lib.device_status(reset=True) == 0
    yield lib
    assert lib.device_status() == 0


def table_in_room(G, n_rot):
    t = torch.zeros(G.rope_table_bytes(1024), dtype=torch.uint8, device="cuda")
    if n_rot:
        G.rope_table(t, n_rot)
    return t


@pytest.mark.parametrize("made", [0, 32, 62, 66, 128])
@pytest.mark.parametrize("T, H, ld", [(1, 3, 0), (300, 2, 0), (5, 2, 131)])
def test_rope(G, T, H, ld, made):
    D = n_rot = 64
    x, pos = torch.randn(T, ld or H * D, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    y = torch.full_like(x, 7.0)
    kw = dict(n_rot=n_rot, ld=ld, ld_dst=ld)
    G.rope(x, T, H, D, pos, table_in_room(G, made), y, **kw)
    assert torch.all(y == 7.0)
    assert G.device_status() == G.ERR_INVALID and G.device_status(reset=True) == G.ERR_INVALID and G.device_status() == G.OK
    G.Graph([G.prepare_rope(x, T, H, D, pos, table_in_room(G, n_rot), y, **kw)]).launch()
    assert not torch.any(y[:, :H * D] == 7.0) and G.device_status() == G.OK


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("T, block", [(3, 16), (300, 16), (300, 2)])
def test_cache_store(G, T, block, fmt, f16):
    """Neither codes, scales nor queries."""
    rng = np.random.default_rng(T)
    H, Hq, D = 2, 5, 64
    table, pages = au.shuffled_table(rng, [T], 16)
    c = au.cache_arrays(rng, fmt, pages, H, 16, D, block, table)
    dc = au.DeviceCache(G, c)
    dt, typ = (torch.float16, G.F16) if f16 else (torch.float32, G.F32)
    q, k, v = (torch.randn(T, h, D, device="cuda").to(dt) for h in (Hq, H, H))
    seq, pos = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    turned = torch.full_like(q, 7.0)
    kw = dict(type=typ, q=q, q_heads=Hq, q_dst=turned)
    for made, n_rot in ((32, 0), (64, 32), (0, 0), (128, 64)):
        G.cache_store(dc.cache, k, v, T, seq, pos, rope=table_in_room(G, made), n_rot=n_rot, **kw)
        assert torch.all(turned == 7.0)
        for name in ("k", "v", "k_scale", "v_scale"):
            assert torch.equal(dc.t[name], dev_tensor(c[name])), name
        assert G.device_status(reset=True) == G.ERR_INVALID and G.device_status() == G.OK
    G.cache_store(dc.cache, k, v, T, seq, pos, rope=table_in_room(G, 64), **kw)
    assert not torch.any(turned == 7.0) and not torch.equal(dc.t["v"], dev_tensor(c["v"])) and G.device_status() == G.OK
