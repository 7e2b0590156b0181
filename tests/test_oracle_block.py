"""Pins of oracle/block.py: hand cases, a direct loop, and central differences
of every gradient in float64."""
import math

import numpy as np
import pytest

from oracle import block as B

STEP = 1e-5


def differences(f, x):
    """Gradient of the scalar f at x by central differences."""
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = x[i]
        x[i] = keep + STEP
        up = f()
        x[i] = keep - STEP
        g[i] = (up - f()) / (2 * STEP)
        x[i] = keep
    return g


def close(a, b):
    # truncation STEP^2 f''' / 6 and rounding 2^-53 f / STEP are both below 1e-9 here
    assert a.shape == b.shape
    assert np.abs(a - b).max() <= 1e-7 * max(1.0, np.abs(b).max())


def test_norm_by_hand():
    h = np.array([[1.0, 2.0]])
    y = np.array([[3.0, 4.0]])
    out, u = B.block_norm(h, y, w_post=np.array([1.0, 2.0]), gate=np.array([0.5, 0.25]), scale=2.0,
                          eps=0.0, w_pre=np.array([1.0, -1.0]))
    r = 1.0 / math.sqrt(12.5)
    want = np.array([[1.0 + 3.0 * r, 2.0 + 4.0 * r]])       # 2 * 0.5 * 3 r, 2 * 0.25 * 2 * 4 r
    assert np.allclose(out, want, rtol=1e-15)
    s = 1.0 / math.sqrt((want ** 2).sum() / 2)
    assert np.allclose(u, want * s * [1.0, -1.0], rtol=1e-15)
    assert B.block_norm(h, w_pre=np.ones(2), eps=0.0)[0] is h
    assert np.array_equal(B.block_norm(h, y, y2=y, scale=0.5)[0], h + y)


def test_activations():
    for g in (-3.0, -0.5, 0.0, 0.7, 4.0):
        f, _ = B.act(np.array(g), "silu")
        assert f == pytest.approx(g / (1.0 + math.exp(-g)), rel=1e-15)
        # the tanh formula stays within 5e-4 of the Gaussian's
        f, _ = B.act(np.array(g), "gelu_tanh")
        assert f == pytest.approx(0.5 * g * (1.0 + math.erf(g / math.sqrt(2.0))), abs=5e-4)


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_ffn_is_the_loop(kind):
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((3, 4)), [rng.standard_normal((4, 5)) for _ in range(3)]
    want = np.zeros((3, 4))
    for t in range(3):
        for n in range(5):
            g = sum(x[t, k] * w[0][k, n] for k in range(4))
            u = sum(x[t, k] * w[1][k, n] for k in range(4))
            for o in range(4):
                want[t, o] += float(B.act(np.array(g), kind)[0]) * u * w[2][o, n]
    assert np.allclose(B.shared_ffn(x, w, kind), want, rtol=1e-12, atol=1e-13)
    assert np.allclose(B.shared_ffn(x, w, kind, add=x), want + x, rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_ffn_gradients_are_differences(kind):
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((3, 4)), [rng.standard_normal((4, 5)) for _ in range(3)]
    dy = rng.standard_normal((3, 4))
    f = lambda: float((dy * B.shared_ffn(x, w, kind)).sum())
    dx, dw = B.shared_ffn_bwd(x, dy, w, kind)
    close(dx, differences(f, x))
    for a, b in zip(dw, w):
        close(a, differences(f, b))


@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
def test_norm_gradients_are_differences(gate, post, pre):
    rng = np.random.default_rng(3)
    n = rng.standard_normal
    T, W = 3, 5
    h, y, y2 = n((T, W)), n((T, W)), n((T, W))
    v = dict(gate=None if gate is None else n({"channel": (W,), "token": (T, 1),
                                              "full": (T, W)}[gate]),
             w_post=n(W) if post else None, w_pre=n(W) if pre else None)
    dh, du = n((T, W)), n((T, W)) if pre else None

    def f():
        out, u = B.block_norm(h, y, y2, scale=0.7, eps=1e-3, **v)
        return float((dh * out).sum() + (0.0 if u is None else (du * u).sum()))

    behind = B.block_norm(h, y, y2, scale=0.7, eps=1e-3, **v)[0]
    dres, dy, *dw = B.block_norm_bwd(behind, dh, du, y, y2, scale=0.7, eps=1e-3, **v)
    close(dres, differences(f, h))
    close(dy, differences(f, y))
    close(dy, differences(f, y2))
    for got, name in zip(dw, ("gate", "w_post", "w_pre")):
        assert (got is None) == (v[name] is None)
        if got is not None:
            close(got, differences(f, v[name]))


def test_norm_alone():
    rng = np.random.default_rng(4)
    h, du, w = rng.standard_normal((2, 6)), rng.standard_normal((2, 6)), rng.standard_normal(6)
    f = lambda: float((du * B.block_norm(h, w_pre=w)[1]).sum())
    dres, dy, dgate, dw_post, dw_pre = B.block_norm_bwd(h, None, du, w_pre=w)
    assert dy is None and dgate is None and dw_post is None
    close(dres, differences(f, h))
    close(dw_pre, differences(f, w))
