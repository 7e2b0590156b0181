"""The bounds of shared_ffn_norms against roundings taken on the host: they hold, and a lost token,
column of H' or split's edge is past them."""
import numpy as np
import pytest
import torch

from oracle import block as B
from shared_ffn_norms import results


def rounded(a):
    return torch.from_numpy(a).bfloat16().double().numpy()


def inputs(T, H, Hp, seed=0):
    rng = np.random.default_rng(seed)
    n = lambda *s: rounded(rng.standard_normal(s))
    return n(T, H), n(T, H), [rounded(rng.standard_normal((H, Hp)) * 1.5 / s ** 0.5)
                              for s in (H, H, Hp)]


def operator(x, dy, w, act):
    """The results with Z, dG, dU and themselves rounded to bf16."""
    g, u = x @ w[0], x @ w[1]
    f, df = B.act(g, act)
    dz = dy @ w[2]
    z, dg, du = rounded(f * u), rounded(dz * u * df), rounded(dz * f)
    return {"y": rounded(z @ w[2].T), "dx": rounded(dg @ w[0].T + du @ w[1].T),
            "dWg": rounded(x.T @ dg), "dWu": rounded(x.T @ du), "dWd": rounded(dy.T @ z)}


def of_bound(got, want):
    return {n: float(np.linalg.norm(got[n] - v)) / e for n, (v, e) in want.items()}


@pytest.mark.parametrize("T,H,Hp,act", [(12301, 128, 192, "silu"), (257, 64, 1024, "gelu_tanh")])
def test_bounds_hold_and_see_a_lost_term(T, H, Hp, act):
    x, dy, w = inputs(T, H, Hp)
    want = results(x, dy, w, act)
    for n, r in of_bound(operator(x, dy, w, act), want).items():
        assert 0.5 < r <= 1.0, (n, r)
    # the last token of a split left out of the sums over tokens
    keep = np.arange(T) != T // 2
    lost = of_bound(operator(x[keep], dy[keep], w, act), {n: want[n] for n in ("dWg", "dWu", "dWd")})
    assert min(lost.values()) > 1.0, lost
    # a column of H' left out of the sums over H'
    lost = of_bound(operator(x, dy, [t[:, :-1] for t in w], act), {n: want[n] for n in ("y", "dx")})
    assert min(lost.values()) > 1.0, lost
