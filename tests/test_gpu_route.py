"""gf_route on the GPU against the fp64 oracle: the choice is equal everywhere (also where
two keys differ by less than 32 bits show), the weights to the rounding of a 32-bit
exponential, sum and division."""

import numpy as np
import pytest

from gpu_util import dev_tensor
from oracle import select as osel

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

SCORES = {"softmax": 0, "sigmoid": 1}


@pytest.fixture(scope="module")
def G(lib):
    yield lib
    assert lib.device_status() == 0


def run(G, l, k, score, bias=None, ld=None, prepared=False, **kw):
    T, E = l.shape
    ld = ld or E
    buf = np.full((T, ld), 1e9, dtype=np.float32)
    buf[:, :E] = l
    ids = torch.full((T * k + 8,), -77, dtype=torch.int32, device="cuda")
    w = torch.full((T * k + 8,), -77.0, device="cuda")
    lt, bt = dev_tensor(buf), None if bias is None else dev_tensor(bias)
    args = (lt, T, E, k, ids, w)
    opts = dict(score=SCORES[score], bias=bt, ld=ld, **kw)
    if prepared:
        call = G.prepare_route(*args, **opts)
        graph = G.Graph([call])
        graph.launch()
    else:
        G.route(*args, **opts)
    torch.cuda.synchronize()
    assert torch.all(ids[T * k:] == -77) and torch.all(w[T * k:] == -77.0)
    return ids[:T * k].view(T, k).cpu().numpy(), w[:T * k].view(T, k).cpu().numpy()


def check(G, l, k, score, bias=None, prepared=False, **kw):
    ids, w = run(G, l, k, score, bias, prepared=prepared, **kw)
    okw = {a: b for a, b in kw.items() if a != "ld"}
    want_ids, want_w = osel.route(l, k, score=score, bias=bias, **okw)
    assert np.array_equal(ids, want_ids)
    # 2^-24 a rounding: the exponential and its argument (its size in units), the sum (its
    # terms in a tree of at most 32 + 5 adds), two divisions or products
    fin = np.where(np.isfinite(l), np.abs(l.astype(np.float64)), 0.0)
    span = np.minimum(2 * fin.max(axis=1, initial=0.0), 200.0)[:, None]
    tol = 2.0 ** -24 * (60 + 3 * span) * np.abs(want_w) + 1e-37
    assert np.all(np.abs(w - want_w) <= tol), float(np.max(np.abs(w - want_w) / tol))
    return ids, w


def logits(T, E, seed, spread=1.5):
    return (np.random.default_rng(seed).standard_normal((T, E)) * spread).astype(np.float32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T, E, k", [(1, 1, 1), (1, 2, 2), (3, 8, 2), (1, 128, 8), (257, 128, 8), (33, 60, 4),
                                     (7, 32, 32), (65, 257, 12), (9, 512, 6), (5, 1000, 32), (300, 1024, 8)])
def test_plain(G, T, E, k, score):
    check(G, logits(T, E, 1), k, score, norm=True, scale=2.5)
    check(G, logits(T, E, 2), k, score, norm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T, E, k", [(1, 128, 8), (1025, 256, 8), (61, 60, 4), (17, 1024, 32)])
def test_bias(G, T, E, k, score):
    b = (np.random.default_rng(5).standard_normal(E) * 0.05).astype(np.float32)
    check(G, logits(T, E, 3), k, score, bias=b)


@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T, E, k, g, keep", [(1, 256, 8, 8, 4), (700, 256, 8, 8, 3), (33, 60, 5, 6, 2),
                                              (9, 96, 3, 32, 7), (4, 8, 4, 8, 4), (130, 160, 6, 8, 8)])
def test_groups(G, T, E, k, g, keep, score, top):
    b = (np.random.default_rng(6).standard_normal(E) * 0.05).astype(np.float32)
    l = logits(T, E, 4)
    check(G, l, k, score, bias=b, n_group=g, topk_group=keep, group_top=top)
    check(G, l, k, score, n_group=g, topk_group=keep, group_top=top, norm=False)


def test_ties_go_to_the_lowest_index(G):
    l = np.zeros((3, 40), dtype=np.float32)
    l[1, 1::2] = -0.0
    l[2] = np.repeat([1.0, 3.0, 2.0, 3.0], 10)
    for bias in (None, np.zeros(40, dtype=np.float32)):
        for score in ("softmax", "sigmoid"):
            ids, _ = check(G, l, 12, score, bias=bias)
            assert ids[0].tolist() == list(range(12)) and ids[1].tolist() == list(range(12))
            assert ids[2].tolist() == list(range(10, 20)) + [30, 31]
    check(G, l, 4, "sigmoid", bias=np.zeros(40, dtype=np.float32), n_group=4, topk_group=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_keys_are_told_apart_in_64_bits(G, score):
    """Keys whose difference is far below a 32-bit rounding: experts e and e + 1 swap logit
    and bias contributions, so that only the exact sum orders them."""
    rng = np.random.default_rng(8)
    E, T = 64, 96
    l = np.zeros((T, E), dtype=np.float32)
    l[:] = rng.standard_normal((T, 1)).astype(np.float32)  # equal scores per row, then one ulp apart
    up = rng.random((T, E)) < 0.5
    l = np.where(up, np.nextafter(l, np.float32(10)), l).astype(np.float32)
    b = (0.5 + rng.integers(-3, 4, E) * 2.0 ** -25).astype(np.float32)
    check(G, l, 8, score, bias=b)
    check(G, l, 4, score, bias=b, n_group=8, topk_group=3)
    check(G, l, 4, score, n_group=8, topk_group=3)


def test_masked_and_extreme_logits(G):
    low = np.finfo(np.float32).min
    l = logits(12, 48, 9)
    l[0] = -np.inf
    l[1] = np.nan
    l[2, 5:] = -np.inf
    l[3, :] = low
    l[4, 7:] = low
    l[5, 3] = np.inf
    l[6, 3:5] = np.inf
    l[7, :] = -200.0
    l[7, 4] = -150.0
    l[8, ::2] = np.nan
    l[9, :] = 90.0
    l[10, :] = -90.0 - np.arange(48, dtype=np.float32)
    for score in ("softmax", "sigmoid"):
        for norm in (True, False):
            ids, w = check(G, l, 8, score, norm=norm)
            assert np.all(ids[:2] == -1) and np.all(w[:2] == 0.0) and np.all(ids[2, 5:] == -1)
        check(G, l, 8, score, n_group=6, topk_group=2)
    b = np.zeros(48, dtype=np.float32)
    b[10] = -np.inf
    b[11] = np.nan
    ids, _ = check(G, l, 8, "sigmoid", bias=b)
    assert not np.isin(ids, (10, 11)).any()


def test_row_stride_and_repeat(G):
    l = logits(37, 60, 10)
    a = check(G, l, 4, "softmax", ld=77)
    b = check(G, l, 4, "softmax", ld=77, prepared=True)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1].view(np.uint32), b[1].view(np.uint32))


def test_other_stream(G):
    l = dev_tensor(logits(64, 128, 11))
    ids, w = torch.empty(64, 8, dtype=torch.int32, device="cuda"), torch.empty(64, 8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        G.route(l, 64, 128, 8, ids, w)
    s.synchronize()
    want, _ = osel.route(l.cpu().numpy(), 8)
    assert np.array_equal(ids.cpu().numpy(), want)
