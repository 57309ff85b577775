"""gf_rope_table and gf_rope on the GPU against the fp64 oracle."""

from decimal import Decimal, getcontext

import numpy as np
import pytest

import attend_util as au
from gpu_util import dev_tensor
from oracle import attend as oatt

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

LAYOUT = {"halves": 0, "pairs": 1}
KINDS = {"plain": 0, "linear": 1, "ramp": 2, "bands": 3}


@pytest.fixture(scope="module")
def G(lib):
    yield lib
    assert lib.device_status() == 0


def table_of(G, n_rot, **kw):
    kw = dict(kw)
    if "kind" in kw:
        kw["kind"] = KINDS[kw["kind"]]
    t = torch.empty(G.rope_table_bytes(n_rot), dtype=torch.uint8, device="cuda")
    G.rope_table(t, n_rot, **kw)
    return t


def tolerance(x, f16, m, angle=0.0):
    """A pair's sizes times: cosine and sine 2 units each and pi 2^-25 of the angle's own rounding to
    32 bits, the products and the sum 3 units, m's rounding one; `angle`: what the 64-bit angle is off."""
    a = np.abs(x).max(axis=-1, keepdims=True)
    b = 2 * a * m * (au.U * 9 + np.pi * 2.0 ** -25 + angle)
    return b + (a * 2 * m * au.HALF + 2.0 ** -25 if f16 else 0.0)


def run(G, x, pos, n_rot, layout, table, f16=False, ld=0, ld_dst=0, at=0, inplace=False, prepared=False):
    T, H, D = x.shape
    dt = torch.float16 if f16 else torch.float32
    w = ld or H * D
    xs = torch.full((at + T * w,), 55.0, dtype=dt, device="cuda")
    rows = xs[at:].view(T, w)
    rows[:, :H * D] = dev_tensor(x.reshape(T, -1)).to(dt)
    wd = w if inplace else (ld_dst or H * D)
    out = xs if inplace else torch.full((at + T * wd,), -77.0, dtype=dt, device="cuda")
    p = dev_tensor(np.asarray(pos, dtype=np.int32))
    args = (xs[at:], T, H, D, p, table, out[at:])
    kw = dict(n_rot=n_rot, layout=LAYOUT[layout], type=G.F16 if f16 else G.F32, ld=ld, ld_dst=ld if inplace else ld_dst)
    if prepared:
        G.Graph([G.prepare_rope(*args, **kw)]).launch()
    else:
        G.rope(*args, **kw)
    torch.cuda.synchronize()
    got = out[at:].view(T, wd)
    rest = got[:, H * D:]
    assert torch.all(rest == (55.0 if inplace else -77.0)) and torch.all(out[:at] == (55.0 if inplace else -77.0))
    return got[:, :H * D].view(T, H, D).double().cpu().numpy(), rows


# T, H, D, n_rot
SHAPES = [(1, 1, 2, 2), (1, 32, 128, 128), (3, 5, 80, 40), (2, 3, 7, 4), (61, 25, 80, 32), (300, 3, 64, 64), (5, 2, 256, 64),
          (9, 40, 128, 128), (4, 1, 96, 20), (2, 2, 1024, 1024), (17, 7, 16, 6)]


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("T, H, D, n_rot", SHAPES)
def test_rope(G, T, H, D, n_rot, layout, f16):
    rng = np.random.default_rng(T + D)
    x = rng.standard_normal((T, H, D)).astype(np.float16 if f16 else np.float32).astype(np.float64)
    pos = rng.integers(-100000, 1 << 24, T)
    pos[0] = 0
    got, _ = run(G, x, pos, n_rot, layout, table_of(G, n_rot), f16)
    want = oatt.rope(x, pos, oatt.freqs(n_rot), layout=layout)
    # both sides' 64-bit frequencies: 2^-48 of an angle below 2^24
    assert np.all(np.abs(got - want) <= tolerance(x, f16, 1.0, 2.0 ** -24))
    assert np.array_equal(got[..., n_rot:], x[..., n_rot:])


@pytest.mark.parametrize("kw", [dict(kind="linear", factor=4.0), dict(kind="ramp", factor=16.0, span=8192, base=500000.0),
                                dict(kind="ramp", factor=2.0, span=100, fast=8.0, slow=2.0), dict(kind="ramp", factor=0.5, span=4096),
                                dict(kind="bands", factor=8.0, span=8192, fast=4.0, slow=1.0, base=500000.0),
                                dict(magnitude=0.25), dict(kind="ramp", factor=4.0, span=4096, magnitude=1.0)])
@pytest.mark.parametrize("n_rot", [2, 64, 128])
def test_scaled(G, n_rot, kw):
    rng = np.random.default_rng(n_rot)
    x = rng.standard_normal((33, 2, 128)).astype(np.float32).astype(np.float64)
    pos = rng.integers(0, 1 << 20, 33)
    okw = {k: v for k, v in kw.items() if k != "magnitude"}
    m = oatt.magnitude(kw.get("kind", "plain"), kw.get("factor", 1.0), kw.get("magnitude", 0.0))
    got, _ = run(G, x, pos, n_rot, "halves", table_of(G, n_rot, **kw))
    want = oatt.rope(x, pos, oatt.freqs(n_rot, **okw), m)
    assert np.all(np.abs(got - want) <= tolerance(x, False, m, 2.0 ** -26))


def test_divisors(G):
    d = np.linspace(1.0, 40.0, 32).astype(np.float32)
    x = np.random.default_rng(1).standard_normal((5, 1, 64)).astype(np.float32).astype(np.float64)
    pos = [0, 1, 1000, 65536, 200000]
    got, _ = run(G, x, pos, 64, "pairs", table_of(G, 64, divisors=dev_tensor(d)))
    assert np.all(np.abs(got - oatt.rope(x, pos, oatt.freqs(64, divisors=d), layout="pairs")) <= tolerance(x, False, 1.0, 2.0 ** -26))


def test_farthest_positions(G):
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    n = 32
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 123456789]
    x = np.zeros((4, 1, 64))
    x[:, 0, :n] = 1.0
    got, _ = run(G, x, pos, 64, "halves", table_of(G, 64))
    ln = Decimal(10000).ln()
    for t, p in enumerate(pos):
        ang = [float((Decimal(p) * (-ln * i / n).exp()) % (2 * pi)) for i in range(n)]
        # the frequency's 64-bit arithmetic: 2^-49 of an angle below 2^31
        tol = 2 * (au.U * 9 + np.pi * 2.0 ** -25 + 2.0 ** -18)
        assert np.all(np.abs(got[t, 0, :n] - np.cos(ang)) <= tol) and np.all(np.abs(got[t, 0, n:] - np.sin(ang)) <= tol)
        assert abs(got[t, 0, 0] - np.cos(ang[0])) <= 2 * (au.U * 9 + np.pi * 2.0 ** -25 + 2.0 ** -20)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("ld, ld_dst, at", [(0, 0, 0), (700, 0, 0), (643, 641, 0), (648, 656, 4), (640, 640, 1), (644, 0, 2)])
def test_strides_and_alignment(G, ld, ld_dst, at, f16):
    rng = np.random.default_rng(ld + at)
    x = rng.standard_normal((7, 5, 128)).astype(np.float16 if f16 else np.float32).astype(np.float64)
    pos = rng.integers(0, 5000, 7)
    table = table_of(G, 96)
    want, _ = run(G, x, pos, 96, "halves", table, f16)
    got, src = run(G, x, pos, 96, "halves", table, f16, ld, ld_dst, at)
    assert np.array_equal(got, want)
    assert np.array_equal(src[:, :640].double().cpu().numpy(), x.reshape(7, -1))
    inplace, _ = run(G, x, pos, 96, "halves", table, f16, ld, ld, at, inplace=True)
    assert np.array_equal(inplace, want)
    again, _ = run(G, x, pos, 96, "halves", table, f16, ld, ld_dst, at, prepared=True)
    assert np.array_equal(again, want)


def test_inverse_and_not_finite(G):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 2, 64)).astype(np.float32).astype(np.float64)
    pos = np.array([0, 5, 77, 4096, 100000, 2 ** 31 - 1])
    table = table_of(G, 64)
    y, _ = run(G, x, pos, 64, "pairs", table)
    back, _ = run(G, y, -pos, 64, "pairs", table)
    assert np.all(np.abs(back - x) <= 2 * tolerance(x, False, 1.0))
    x[2, 1, 10] = np.nan
    x[3, 0, 63] = np.inf
    got, _ = run(G, x, pos, 64, "pairs", table)
    bad = ~np.isfinite(got)
    assert bad[2, 1, 10:12].all() and bad[3, 0, 62:].all() and bad.sum() == 4
