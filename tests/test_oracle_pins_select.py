"""Pins for the oracle of routing, the chosen experts' product and low-rank adapters: hand
worked values, closed forms, brute force over subsets; and planted mistakes that a pin
has to catch."""

import itertools

import numpy as np
import pytest

from oracle import gemv, quant, select

F32 = quant.WTYPE_F32


def _raw(a):
    return np.ascontiguousarray(a, dtype="<f4").reshape(-1).view(np.uint8)


def test_route_worked_softmax():
    # e^l = 1, 2, 4, 1: softmax 1/8, 2/8, 4/8, 1/8
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    ids, w = select.route(l, 3, norm=False)
    assert ids.tolist() == [[2, 1, 0]]  # the tie of 0 and 3 goes to 0
    assert np.allclose(w, [[0.5, 0.25, 0.125]], rtol=1e-14)
    _, w = select.route(l, 2, norm=True, scale=3.0)
    assert np.allclose(w, [[2.0, 1.0]], rtol=1e-14)


def test_route_sigmoid_bias_is_for_the_choice_only():
    l = np.array([[0.0, 0.0, np.log(3.0)]])  # scores 1/2, 1/2, 3/4
    ids, w = select.route(l, 2, score="sigmoid", bias=np.array([0.0, 0.5, 0.0]), norm=False)
    assert ids.tolist() == [[1, 2]]
    assert np.allclose(w, [[0.5, 0.75]], rtol=1e-14)


def test_route_groups():
    # keys (sigmoid scores) by group: {.9, .1}, {.6, .6}, {.8, .3}: best sums 1.0, 1.2, 1.1; best maxima .9, .8
    s = np.array([[0.9, 0.1, 0.6, 0.6, 0.8, 0.3]])
    l = np.log(s / (1 - s))
    two = select.route(l, 2, score="sigmoid", n_group=3, topk_group=2, group_top=2)[0]
    one = select.route(l, 2, score="sigmoid", n_group=3, topk_group=2, group_top=1)[0]
    assert two.tolist() == [[4, 2]] and one.tolist() == [[0, 4]]


def test_route_masked_rows():
    l = np.array([[-np.inf, np.nan, -np.inf], [1.0, -np.inf, 2.0]])
    ids, w = select.route(l, 2)
    assert ids[0].tolist() == [-1, -1] and w[0].tolist() == [0.0, 0.0]
    assert ids[1].tolist() == [2, 0] and np.isclose(w[1].sum(), 1.0)


def test_route_is_the_best_subset():
    rng = np.random.default_rng(0)
    l = rng.standard_normal((20, 6))
    b = rng.standard_normal(6) * 0.3
    ids, _ = select.route(l, 3, score="sigmoid", bias=b)
    key = 1.0 / (1.0 + np.exp(-l)) + b
    for t in range(20):
        best = max(itertools.combinations(range(6), 3), key=lambda c: sum(key[t, list(c)]))
        assert sorted(ids[t].tolist()) == list(best)
        assert list(ids[t]) == sorted(best, key=lambda e: -key[t, e])


def test_experts_one_hot_and_sum():
    rng = np.random.default_rng(1)
    E, M, K = 3, 4, 5
    G, U, D = rng.standard_normal((E, M, K)), rng.standard_normal((E, M, K)), rng.standard_normal((E, K, M))
    G, U, D = (a.astype(np.float32).astype(np.float64) for a in (G, U, D))
    x = rng.standard_normal((2, K))
    ids = np.array([[0, 2], [1, -1]])
    w = np.array([[0.25, 0.75], [1.0, 9.0]])

    def ffn(e, v):
        g = G[e] @ v
        return D[e] @ (g / (1 + np.exp(-g)) * (U[e] @ v))

    got, bound = select.experts(_raw(G), _raw(U), F32, _raw(D), F32, E, x, M, K, ids, w)
    assert np.allclose(got[0], 0.25 * ffn(0, x[0]) + 0.75 * ffn(2, x[0]), rtol=1e-12)
    assert np.allclose(got[1], ffn(1, x[1]), rtol=1e-12)  # the id -1 adds nothing
    assert np.all(bound > 0)
    # a planted mistake, the weight inside the activation's product squared, is seen
    assert not np.allclose(got[0], 0.0625 * ffn(0, x[0]) + 0.75 * ffn(2, x[0]), rtol=1e-6)


@pytest.mark.parametrize("epi", range(5))
def test_lora_is_the_merged_matrix(epi):
    rng = np.random.default_rng(2)
    M, K, r, n = 6, 8, 3, 2
    W = rng.standard_normal((M, K)).astype(np.float32)
    A, B = rng.standard_normal((n, r, K)), rng.standard_normal((n, M, r))
    x = rng.standard_normal((3, K))
    aux = rng.standard_normal((3, M))
    s = np.array([0.5, 2.0])
    got, _ = select.lora(_raw(W), F32, x, M, K, epi, aux, A, B, [1, -1, 0], s)
    for c, a in enumerate([1, -1, 0]):
        Wm = W.astype(np.float64) + (s[a] * B[a] @ A[a] if a >= 0 else 0.0)
        want = gemv.apply_epilogue((Wm @ x[c])[None], epi, aux[c][None])[0]
        assert np.allclose(got[c], want, rtol=1e-12)
