"""What surrounds the expert path inside one transformer block: the norms with
gate and residual scale, and the shared expert's gated feed-forward block,
forward and backward.  TEST INFRASTRUCTURE ONLY.

The pages leave these to the framework (MoonEP README, MoonshotAI/MoonEP
mirror, "Usage > Integration"); they are written here from their definitions in
float64 and pinned by finite differences (tests/test_oracle_block.py).  Arrays
are float64 throughout; a None stands for an input that is not there.
"""
import math

import numpy as np


def rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def block_norm(h, y=None, y2=None, gate=None, w_post=None, w_pre=None, scale=1.0, eps=1e-6):
    """(h', u): gate broadcasts over [T,W]."""
    out = h
    if y is not None:
        n = y if y2 is None else y + y2
        if w_post is not None:
            n = n * rstd(n, eps) * w_post
        if gate is not None:
            n = n * gate
        out = h + scale * n
    return out, None if w_pre is None else out * rstd(out, eps) * w_pre


def _norm_bwd(x, w, d, eps):
    """(dx, dw) of x rstd(x) w for the gradient d."""
    r = rstd(x, eps)
    hat = x * r
    v = d * w
    return r * (v - hat * (v * hat).mean(-1, keepdims=True)), (d * hat).sum(0)


def block_norm_bwd(h, dh, du=None, y=None, y2=None, gate=None, w_post=None, w_pre=None, scale=1.0,
                   eps=1e-6):
    """(dres, dy, dgate, dw_post, dw_pre); h is the stream behind the block."""
    d = np.zeros_like(h) if dh is None else dh
    dw_pre = dw_post = dgate = dy = None
    if w_pre is not None:
        dx, dw_pre = _norm_bwd(h, w_pre, du, eps)
        d = d + dx
    if y is not None:
        a = y if y2 is None else y + y2
        n = a if w_post is None else a * rstd(a, eps) * w_post
        dn = scale * d
        if gate is not None:
            t = dn * n
            dgate = t if gate.shape == t.shape else \
                t.sum(0) if gate.ndim == 1 else t.sum(-1, keepdims=True)
            dn = dn * gate
        dy = dn
        if w_post is not None:
            dy, dw_post = _norm_bwd(a, w_post, dn, eps)
    return d, dy, dgate, dw_post, dw_pre


def act(g, kind):
    """(f, f'): silu, or gelu by the tanh formula."""
    if kind == "silu":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-g))
        return g * s, s + g * s * (1.0 - s)
    k = math.sqrt(2.0 / math.pi)
    t = np.tanh(k * (g + 0.044715 * g ** 3))
    return (0.5 * g * (1.0 + t),
            0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g * g))


def shared_ffn(x, w, kind="silu", add=None):
    """Y = (act(X Wg) * (X Wu)) Wd^T (+ add); w = (Wg, Wu, Wd), each [H,H']."""
    z = act(x @ w[0], kind)[0] * (x @ w[1])
    y = z @ w[2].T
    return y if add is None else y + add


def shared_ffn_bwd(x, dy, w, kind="silu"):
    """(dX, (dWg, dWu, dWd))."""
    g, u = x @ w[0], x @ w[1]
    f, df = act(g, kind)
    dz = dy @ w[2]
    dg, du = dz * u * df, dz * f
    return dg @ w[0].T + du @ w[1].T, (x.T @ dg, x.T @ du, dy.T @ (f * u))
