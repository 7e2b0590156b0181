"""Pins of oracle/training.py: the router's gradient and the combine's by
central differences, the orthogonalisation by the singular values."""
import numpy as np
import pytest

import oracle
from oracle import training as T

FORMS = [(s, n) for s in ("softmax", "sigmoid") for n in (True, False)]


@pytest.mark.parametrize("score,normalize", FORMS)
@pytest.mark.parametrize("bias", [False, True])
def test_route_by_hand(score, normalize, bias):
    x = np.array([[0.5, 2.0, 2.0, -1.0, 1.0], [3.0, 0.0, 0.0, 0.0, 0.0]])
    b = np.array([0.0, 0.0, 0.0, 5.0, 0.0]) if bias else None
    ids, w = T.route(x, 3, b, score, normalize, 2.0)
    assert ids.tolist() == ([[3, 1, 2], [3, 0, 1]] if bias else [[1, 2, 4], [0, 1, 2]])
    p = np.exp(x) / np.exp(x).sum(1, keepdims=True) if score == "softmax" else 1 / (1 + np.exp(-x))
    for r in range(2):
        q = p[r, ids[r]]
        assert np.allclose(w[r], 2.0 * (q / q.sum() if normalize else q), rtol=1e-14)


@pytest.mark.parametrize("score,normalize", FORMS)
def test_closed_experts_come_last_with_weight_zero(score, normalize):
    inf = np.inf
    x = np.array([[-inf, 1.0, -inf, 0.5], [-inf, -inf, -inf, -inf]])
    for bias in (None, np.array([9.0, 0.0, 0.0, 0.0])):
        ids, w = T.route(x, 3, bias, score, normalize)
        assert ids.tolist() == [[1, 3, 0], [0, 1, 2]]
        assert w[0, 2] == 0 and np.all(w[1] == 0) and np.all(np.isfinite(w))
        d = T.route_bwd(x, ids, np.ones((2, 3)), score, normalize)
        assert np.all(np.isfinite(d)) and np.all(d[1] == 0) and np.all(d[0, [0, 2]] == 0)


@pytest.mark.parametrize("score,normalize", FORMS)
def test_route_gradient_against_differences(score, normalize):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 9))
    ids, _ = T.route(x, 4, None, score, normalize, 1.7)
    c = rng.standard_normal(ids.shape)

    def loss(v):
        p = T.scores(v, score)
        q = np.take_along_axis(p, ids, axis=-1)
        w = 1.7 * (q / q.sum(-1, keepdims=True) if normalize else q)
        return (c * w).sum()

    got = T.route_bwd(x, ids, c, score, normalize, 1.7)
    h = 1e-5
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        want = (loss(x + e) - loss(x - e)) / (2 * h)
        # truncation h^2/6 of a third derivative of order one, cancellation 2^-53 / h
        assert abs(got[i] - want) < 1e-9


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(5)
    R, S, K, E, W = 2, 5, 2, 4, 6
    topk = np.array([[rng.permutation(E)[:K] for _ in range(S)] for _ in range(R)])
    p = oracle.plan(topk, E, E // R, 4)
    bf = lambda shape: oracle.f32_to_bf16(rng.standard_normal(shape).astype(np.float32))
    dout, y = bf((R, S, W)), bf((R, p.NvS, W))
    rw = rng.random((R, p.NvS)).astype(np.float32)
    dy, drw, _ = T.combine_bwd(p, dout, y, rw)
    c = oracle.bf16_to_f32(dout).astype(np.float64)
    yv = oracle.bf16_to_f32(y).astype(np.float64).reshape(-1, W)
    wv = rw.astype(np.float64).reshape(-1)

    def loss(yv, wv):
        out = (wv[p.dest][..., None] * yv[p.dest]).sum(axis=2)
        return (c * out).sum()

    for r, s, k in np.ndindex(R, S, K):
        slot = p.dest[r, s, k]
        e = np.zeros_like(wv)
        e[slot] = 1e-4                                  # the loss is linear in each
        assert np.isclose((loss(yv, wv + e) - loss(yv, wv - e)) / 2e-4, drw[r, s, k], atol=1e-9)
        got = oracle.bf16_to_f32(dy.reshape(-1, W)[slot])
        assert np.all(np.abs(got - wv[slot] * c[r, s]) <= 2.0 ** -8 * np.abs(wv[slot] * c[r, s]))
    none = np.setdiff1d(np.arange(R * p.NvS), p.dest)
    assert not dy.reshape(-1, W)[none].any()


@pytest.mark.parametrize("rows,cols", [(1, 1), (7, 5), (5, 12)])
def test_orthogonalize_is_a_polynomial_of_the_singular_values(rows, cols):
    g = np.random.default_rng(rows).standard_normal((rows, cols))
    co = [(3.4445, -4.7750, 2.0315)] * 4 + [(2.0, -1.5, 0.5)]
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + 1e-3)
    for a, b, c in co:
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(T.orthogonalize(g, co, 1e-3), (u * s) @ vt, atol=1e-12)
