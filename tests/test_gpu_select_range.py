"""Dynamic range of x, and of the gated values, in the tiled products of gemv_experts and
gemv_lora: outliers on columns whose weights are zero.  Gated on the literal bound of each
product, as tests/test_gpu_int_dot.py gates the single-column kernels; each case asserts the
kernel that its shape takes."""

import numpy as np
import pytest

from decode_gemv_epilogue_gb300 import synth
from gpu_util import assert_within, dev_tensor
from oracle import quant as oquant

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import test_gpu_experts  # noqa: E402
import test_gpu_lora  # noqa: E402
from test_gpu_int_dot import zero_weight_columns  # noqa: E402

F32, F16, Q8, Q4, Q4K = synth.F32, synth.F16, synth.Q8_0, synth.Q4_0, synth.Q4_K
SPIKES = (5, 70, 71, 263)  # 70 and 71 share a block; of Q4_K's sub-blocks 0..3


@pytest.fixture(scope="module")
def G(lib):
    assert lib.device_status(reset=True) == 0
    yield lib
    assert lib.device_status() == 0, "a kernel reported a bounded-wait timeout"


def zero_columns(raw, wt, rows, K, cols):
    if wt in (F32, F16):
        w = raw.copy().view(np.float32 if wt == F32 else np.float16).reshape(rows, K)
        w[:, list(cols)] = 0
        return w.reshape(-1).view(np.uint8)
    return zero_weight_columns(raw, wt, rows, K, cols)


def spiked(x, cols, size):
    """x with spikes of +-size on `cols` in every second row."""
    x = x.copy()
    x[::2, list(cols)] = size * np.where(np.arange(len(cols)) % 2 == 0, 1.0, -1.0)
    return x.astype(np.float32)


# (T, E, k, M, K) and the columns of a group: one, few, one tile, several, the wide kernel
EXPERTS = {
    "one": (1, 4, 3, 256, 512, 1),
    "few": (3, 4, 2, 256, 512, 3),
    "tile": (9, 3, 2, 256, 512, 8),
    "wide": (256, 4, 4, 512, 512, 16),
}


def experts_case(G, wt, kind, seed):
    T, E, k, M, K, cols = EXPERTS[kind]
    if wt in (F32, F16):
        cols = {"tile": 16, "wide": 24}.get(kind, cols)
    c = test_gpu_experts.Case(G, T, E, k, M, K, wt, wt, seed=seed)
    ws = torch.empty(G.experts_workspace(E, T, k, M, K), dtype=torch.uint8, device="cuda")
    path, info = G.plan_experts(c.dev[0], c.dev[1], wt, c.dev[2], wt, E, dev_tensor(c.x), M, K, dev_tensor(c.ids),
                                dev_tensor(c.w), T, k, None, torch.empty(T * K, device="cuda"), ws)
    assert path == 4 and info["cols"] == cols
    return c


def set_raw(c, i, raw):
    c.raw[i], c.dev[i] = raw, dev_tensor(raw)


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("kind", list(EXPERTS))
@pytest.mark.parametrize("size", [1e3, 1e5, 1e6])
def test_experts_outliers_of_x(G, wt, kind, size):
    c = experts_case(G, wt, kind, seed=300)
    for i in (0, 1):
        set_raw(c, i, zero_columns(c.raw[i], wt, c.E * c.M, c.K, SPIKES))
    x = spiked(c.x, SPIKES, size)
    y, b = c.want(x=x)
    assert_within(c.run(x=x), y, b, "spikes of %g" % size)


def gated_spikes(c, wt, size):
    """Weights whose gated values hold spikes of about `size` on the columns SPIKES[:3] of the down
    product, which are zero there."""
    cols = SPIKES[:3]
    c.x[:, 0] = 1.0  # the up rows of the spikes take their size from this column
    set_raw(c, 2, zero_columns(c.raw[2], wt, c.E * c.K, c.M, cols))
    rb = oquant.row_bytes(wt, c.K)
    for i in (0, 1):
        raw = c.raw[i].copy().reshape(c.E, c.M, rb)
        for m in cols:
            if wt == F32:
                raw[:, m].view(np.float32)[:, 0] = size if i else 3.0
            elif wt == F16:
                raw[:, m].view(np.float16)[:, 0] = min(size, 6e4) if i else 3.0
            else:  # the first block's scale; its first code far from zero
                d = np.frombuffer(np.float16(min(size / 4, 6e4) if i else 2.0).tobytes(), np.uint8)
                raw[:, m, 0:2] = d
                if wt == Q8:
                    raw[:, m, 2:34] = 0
                    raw[:, m, 2] = 100 if i else 2
                elif wt == Q4:
                    raw[:, m, 2:18] = 0x88
                    raw[:, m, 2] = 0x8F if i else 0x8A
                else:
                    raw[:, m, 2:144] = 0  # no mins, scales 1 of sub-block 0 only
                    raw[:, m, 4] = 1
                    raw[:, m, 16] = 0x0F if i else 0x02
        set_raw(c, i, raw.reshape(-1))


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("kind", list(EXPERTS))
@pytest.mark.parametrize("size", [1e3, 1e5, 1e6])
def test_experts_outliers_of_the_gated_values(G, wt, kind, size):
    c = experts_case(G, wt, kind, seed=310)
    gated_spikes(c, wt, size)
    y, b = c.want()
    assert_within(c.run(), y, b, "gated spikes of %g" % size)


# (N, M, K) and the columns of a group
LORA = {"few": (3, 16384, 2816, 3), "tile": (8, 8200, 2048, 8), "two": (40, 300, 512, 8), "wide": (250, 4500, 512, 16)}


def lora_case(G, wt, kind, seed):
    N, M, K, cols = LORA[kind]
    if wt in (F32, F16):
        if kind != "two":
            pytest.skip("plain rows have one kernel here")
        N, M, K, cols = 40, 2100, 512 if wt == F32 else 480, 16  # (F16 rows of whole 64s go to another)
    c = test_gpu_lora.Case(G, N, M, K, wt, 3, 8, F16, seed=seed)
    path, info = G.plan_lora(c.Wd, wt, dev_tensor(c.x), M, K, 0, None, torch.empty(N * M, device="cuda"), c.Ad, c.Bd, F16,
                             c.n, c.r, dev_tensor(c.ids), None,
                             torch.empty(G.lora_workspace(N, M, K, c.r, c.n), dtype=torch.uint8, device="cuda"), ncols=N)
    assert path == 4 and info["cols"] == cols
    return c


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("kind", list(LORA))
@pytest.mark.parametrize("size", [1e3, 1e5, 1e6])
def test_lora_outliers_of_x(G, wt, kind, size):
    c = lora_case(G, wt, kind, seed=320)
    c.raw = zero_columns(c.raw, wt, c.M, c.K, SPIKES)
    c.Wd = dev_tensor(c.raw)
    c.A[:, :, list(SPIKES)] = 0
    c.Ad = dev_tensor(c.A)
    x = spiked(c.x, SPIKES, size)
    y, b = c.want(2, x=x)
    assert_within(c.run(2, x=x), y, b, "spikes of %g" % size)


# ----------------------------------------------------------------------------- infinities and NaN

def signed(wt, sign, seed):
    """Raw weights of a format, of sign +1 or -1 where `sign` [rows, K] says so (0: any)."""
    g = np.random.default_rng(seed)
    rows, K = sign.shape
    if wt in (F32, F16):
        w = g.standard_normal((rows, K))
        w = np.where(sign == 0, w, (np.abs(w) + 0.01) * sign) * 0.05
        return w.astype(np.float32 if wt == F32 else np.float16).view(np.uint8).reshape(-1)
    if wt == Q8:
        c = g.integers(-127, 128, (rows, K))
        c = np.where(sign == 0, c, np.maximum(np.abs(c), 1) * sign)
        return synth.pack_q8_0(c, g.uniform(0.0005, 0.002, (rows, K // 32)).astype(np.float16)).reshape(-1)
    if wt == Q4:
        c = g.integers(0, 16, (rows, K))
        c = np.where(sign > 0, np.maximum(c, 9), np.where(sign < 0, np.minimum(c, 7), c))
        return synth.pack_q4_0(c, g.uniform(0.005, 0.02, (rows, K // 32)).astype(np.float16)).reshape(-1)
    c = g.integers(0, 16, (rows, K))  # w = d (sc q - m): scales over 32, mins 1..20
    c = np.where(sign > 0, np.maximum(c, 1), np.where(sign < 0, 0, c))
    d = g.uniform(1e-4, 4e-4, (rows, K // 256)).astype(np.float16)
    return synth.pack_q4_k(c, g.integers(32, 64, (rows, K // 256, 8)), g.integers(1, 21, (rows, K // 256, 8)), d, d).reshape(-1)


def assert_classes(got, want):
    assert np.array_equal(np.isnan(got), np.isnan(want)), "NaN pattern differs"
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(got), inf), "Inf pattern differs"
    assert np.array_equal(got[inf], want[inf]), "sign of an infinity differs"


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("kind", list(EXPERTS))
def test_experts_infinite_x(G, wt, kind):
    """Gate and up weights positive on one column, where x is +inf: every gated value is +inf, and
    the outputs are +inf, -inf or NaN by the signs of the down rows (all +, all -, mixed)."""
    c = experts_case(G, wt, kind, seed=330)
    sign = np.zeros((c.E * c.M, c.K), dtype=int)
    sign[:, 37] = 1
    for i in (0, 1):
        set_raw(c, i, signed(wt, sign, 331 + i))
    sign = np.zeros((c.E * c.K, c.M), dtype=int)
    sign[0::3], sign[1::3] = 1, -1
    assert c.K % 3 != 0  # rows change their class from expert to expert, so keep them apart
    sign = np.concatenate([sign[:c.K]] * c.E)
    set_raw(c, 2, signed(wt, sign, 333))
    c.w += 0.1
    x = c.x.copy()
    x[0, 37] = np.inf
    if c.T > 2:
        x[2, 37], x[c.T - 1, 38] = np.inf, -np.inf
    G.repair_count(reset=True)
    got = c.run(x=x)
    assert G.repair_count(reset=True) > 0
    with np.errstate(invalid="ignore", over="ignore"):
        want, b = c.want(x=x)
    assert np.any(want[0] == np.inf) and np.any(want[0] == -np.inf) and np.any(np.isnan(want[0]))
    assert_classes(got, want)
    fin = np.isfinite(want).all(axis=1)
    assert_within(got[fin], want[fin], b[fin])
    c.run()
    assert G.repair_count() == 0


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("kind", list(LORA))
def test_lora_non_finite_x(G, wt, kind):
    c = lora_case(G, wt, kind, seed=340)
    c.raw = zero_columns(c.raw, wt, c.M, c.K, (5,)) if wt != Q4K else c.raw
    c.Wd = dev_tensor(c.raw)
    x = c.x.copy()
    c.ids[:3] = -1
    x[0, 37], x[1, 5], x[2, 3] = np.inf, -np.inf, np.nan
    if c.N > 3:
        c.ids[5:8] = -1
        x[6, 300] = -np.inf
        x[7, 37], x[7, 300] = np.inf, -np.inf
    for epi in (0, 1):
        G.repair_count(reset=True)
        got = c.run(epi, x=x)
        assert G.repair_count(reset=True) > 0
        with np.errstate(invalid="ignore", over="ignore"):
            want, b = c.want(epi, x=x)
        assert_classes(got, want)
        fin = np.isfinite(want)
        with np.errstate(invalid="ignore"):
            assert_within(got[fin], want[fin], np.where(np.isfinite(b), b, 1e-6)[fin])
    c.run(0)
    assert G.repair_count() == 0


# ----------------------------------------------------------------------------- values that two f16 parts cannot carry

@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("kind", list(EXPERTS))
@pytest.mark.parametrize("size", [1e7, 1e9, 1e13, 1e25])
def test_experts_far_outliers_of_x(G, wt, kind, size):
    c = experts_case(G, wt, kind, seed=350)
    for i in (0, 1):
        set_raw(c, i, zero_columns(c.raw[i], wt, c.E * c.M, c.K, SPIKES))
    x = spiked(c.x, SPIKES, size)
    y, b = c.want(x=x)
    G.repair_count(reset=True)
    assert_within(c.run(x=x), y, b, "spikes of %g" % size)
    assert G.repair_count(reset=True) > 0
    c.run(x=spiked(c.x, SPIKES, 1e4))
    assert G.repair_count() == 0


@pytest.mark.parametrize("kind", list(EXPERTS))
@pytest.mark.parametrize("wd", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("size", [1e9, 1e12, 1e20])
def test_experts_far_outliers_of_the_gated_values(G, kind, wd, size):
    if kind == "wide" and wd in (F32, F16):
        pytest.skip("no wide kernel of these rows")
    T, E, k, M, K, _ = EXPERTS[kind]
    c = experts_case(G, wd, kind, seed=360)
    # two rows of the up matrix, whose gate is 3, take their value from one element of x alone
    cols = SPIKES[1:3]
    set_raw(c, 2, zero_columns(c.raw[2], wd, E * K, M, cols))
    c.x[:, 300:332] = 0.0
    c.x[::2, 300] = size
    for i in (0, 1):  # x is far above the rest there: zero weights but in those rows
        raw = zero_columns(c.raw[i], wd, E * M, K, range(288, 320))
        rows = raw.reshape(E, M, -1)
        for m in cols:
            one = np.zeros((1, K))
            one[0, 300 if i else 5] = 1.0
            rows[:, m] = one_hot(wd, one)
        set_raw(c, i, rows.reshape(-1))
    c.x[:, 5] = 1.0 if wd in (F32, F16) else 3.0
    y, b = c.want()
    G.repair_count(reset=True)
    assert_within(c.run(), y, b, "gated spikes")
    assert G.repair_count() > 0


def one_hot(wt, w):
    """Raw row of weights that are zero but for one of about 1."""
    K = w.shape[1]
    if wt in (F32, F16):
        return w.astype(np.float32 if wt == F32 else np.float16).view(np.uint8).reshape(-1)
    if wt == Q8:
        return synth.pack_q8_0((w * 100).astype(np.int16), np.full((1, K // 32), 0.01, np.float16)).reshape(-1)
    if wt == Q4:
        return synth.pack_q4_0((w * 7 + 8).astype(np.int16), np.full((1, K // 32), 0.14, np.float16)).reshape(-1)
    z = np.zeros((1, K // 256, 8), dtype=np.int16)
    one = np.full((1, K // 256), 0.01, np.float16)
    return synth.pack_q4_k((w * 10).astype(np.int16), z + 10, z, one, one).reshape(-1)


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("kind", list(LORA))
@pytest.mark.parametrize("size", [1e7, 1e9, 1e13, 1e25])
def test_lora_far_outliers_of_x(G, wt, kind, size):
    c = lora_case(G, wt, kind, seed=370)
    c.raw = zero_columns(c.raw, wt, c.M, c.K, SPIKES)
    c.Wd = dev_tensor(c.raw)
    c.A[:, :, list(SPIKES)] = 0
    c.Ad = dev_tensor(c.A)
    x = spiked(c.x, SPIKES, size)
    y, b = c.want(2, x=x)
    G.repair_count(reset=True)
    assert_within(c.run(2, x=x), y, b, "spikes of %g" % size)
    assert G.repair_count(reset=True) > 0
    c.run(2, x=spiked(c.x, SPIKES, 1e4))
    assert G.repair_count() == 0


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4])
@pytest.mark.parametrize("size", [1e3, 1e4, 1e5, 3e5, 1e6])
def test_outliers_in_one_block(G, wt, size):
    """K of one block: nothing else in the row hides what its one outlier costs."""
    c = test_gpu_experts.Case(G, 9, 3, 2, 64, 32, wt, wt, seed=380)
    for i in (0, 1):
        set_raw(c, i, zero_columns(c.raw[i], wt, c.E * c.M, 32, (7,)))
    x = spiked(c.x, (7,), size)
    y, b = c.want(x=x)
    assert_within(c.run(x=x), y, b)


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("case", ["one block", "half", "tiny block", "sparse", "one-hot", "zeros", "cubes"])
def test_uneven_x(G, wt, case):
    """Columns whose blocks differ by many magnitudes, with zero weights on the large ones; and
    columns of few values, which the two parts carry."""
    c = experts_case(G, wt, "tile", seed=390)
    g = np.random.default_rng(391)
    x, large = c.x.astype(np.float64), ()
    if case == "one block":
        x[:, 64:96] *= 1e10
        large = range(64, 96)
    elif case == "half":
        large = [k for k in range(c.K) if k % 256 < 128]
        x[:, large] *= 1e8
    elif case == "tiny block":
        x[:, 64:96] *= 1e-10
    elif case == "sparse":
        x = np.where(g.random(x.shape) < 1 / 64, x, 0.0)
    elif case == "one-hot":
        x = np.where(np.arange(c.K) == np.arange(c.T)[:, None] * 41, x, 0.0)
    elif case == "zeros":
        x[::2] = 0.0
        x[1::2, 5:] = 0.0
    else:
        x = x ** 3
    for i in (0, 1):
        set_raw(c, i, zero_columns(c.raw[i], wt, c.E * c.M, c.K, large) if len(large) else c.raw[i])
    x = x.astype(np.float32)
    y, b = c.want(x=x)
    G.repair_count(reset=True)
    assert_within(c.run(x=x), y, b)
    assert (G.repair_count() > 0) == (case in ("one block", "half"))


@pytest.mark.parametrize("wt", [F32, F16, Q8, Q4, Q4K])
@pytest.mark.parametrize("kind", list(EXPERTS))
def test_experts_nan_goes_the_ordinary_way(G, wt, kind):
    """Nothing but NaN comes of a NaN, so a token that holds one (and one whose x is infinite ahead of
    the normalisation) costs the batch nothing."""
    c = experts_case(G, wt, kind, seed=400)
    x = c.x.copy()
    x[0, 5] = np.nan
    G.repair_count(reset=True)
    got = c.run(x=x)
    assert np.all(np.isnan(got[0])) and np.all(np.isfinite(got[1:]))
    x[0, 5] = np.inf
    got = c.run(x=x, norm=np.ones(c.K, np.float32))
    assert np.all(np.isnan(got[0])) and np.all(np.isfinite(got[1:]))
    assert G.repair_count() == 0
