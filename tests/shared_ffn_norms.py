"""How far results of the shared expert may be off in their norm, where a bound per element is too wide
to see a lost term.

A rounding to bf16 is off by at most half a step, uniformly within it, so by at most b / sqrt(3) of the
value in root mean square, b = 2^-8; those of Z, dG, dU and of a bf16 result are independent and of
mean zero.  An error's squares then sum to at most b^2 / 3 of the squares of everything that was
rounded, each times the squares of what it is multiplied by.  (Over a binade the mean is b^2 / 5.5, so
about 0.74 of the bound is what to expect.)  fp32 sums are off by some 2^-24 sqrt(K), nothing beside
it.  A token or a column that is lost or taken twice shows as its share of the norm: of T tokens 1 /
sqrt(T), past the bound of b / sqrt(3) up to 190 thousand of them."""
import numpy as np

from oracle import block as B

HALF = 2.0 ** -8
E = 2.0 ** -24


def rms(*squares):
    """b / sqrt(3) times the root of the sum of all squares."""
    return HALF * np.sqrt(sum(float(s.sum()) for s in squares) / 3)


def results(x, dy, w, act, f32=False):
    """{name: (value, bound on the error's norm)} from float64 inputs; f32: weight gradients that are
    not rounded (fp32, added to gradients of 0.5)."""
    g, u = x @ w[0], x @ w[1]
    f, df = B.act(g, act)
    z, dz = f * u, dy @ w[2]
    dg, du = dz * u * df, dz * f
    q = lambda t: t * t
    out = {"y": (z @ w[2].T, (q(z) @ q(w[2]).T,)),
           "dx": (dg @ w[0].T + du @ w[1].T, (q(dg) @ q(w[0]).T, q(du) @ q(w[1]).T)),
           "dWg": (x.T @ dg, (q(x).T @ q(dg),)), "dWu": (x.T @ du, (q(x).T @ q(du),)),
           "dWd": (dy.T @ z, (q(dy).T @ q(z),))}
    bounds = {}
    for name, (v, parts) in out.items():
        if f32 and name.startswith("dW"):
            v = v + 0.5
            bounds[name] = (v, rms(*parts) + E * np.linalg.norm(v))
        else:
            bounds[name] = (v, rms(*parts, q(v)))
    return bounds
