"""Steps of a training iteration around the expert path: the router, the
gradient of the weighted combine, and the orthogonalised direction of a weight
gradient.  TEST INFRASTRUCTURE ONLY.

The pages leave these to the framework (MoonEP README, MoonshotAI/MoonEP
mirror, "API guide": topk_experts_sk and route_weights_sk are dispatch's
inputs, the FFN and autograd are the framework's); they are written here from
their definitions in float64, and pinned by finite differences and by the
singular value decomposition (tests/test_oracle_training.py).
"""
import numpy as np

from .bf16 import bf16_to_f32, f32_to_bf16


def scores(logits, score):
    """Softmax or sigmoid of float64 logits [..., E]; a row whose logits are
    all -inf has scores of zero."""
    x = np.asarray(logits, np.float64)
    with np.errstate(over="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        top = x.max(axis=-1, keepdims=True)
        e = np.exp(x - np.where(np.isneginf(top), 0.0, top))
    s = e.sum(axis=-1, keepdims=True)
    return e / np.where(s == 0, 1.0, s)


def _inverse(t):
    return np.where(t == 0, 0.0, 1.0 / np.where(t == 0, 1.0, t))


def route(logits, K, bias=None, score="softmax", normalize=True, scale=1.0):
    """logits [..., E] -> (ids [..., K] int64, weights [..., K] float64).  The
    choice goes by the logit, or by score + bias; equal ones by ascending id;
    a logit of -inf comes after every other."""
    x = np.asarray(logits, np.float64)
    p = scores(x, score)
    key = x if bias is None else np.where(np.isneginf(x), -np.inf, p + np.asarray(bias, np.float64))
    ids = np.argsort(-key, axis=-1, kind="stable")[..., :K]
    w = np.take_along_axis(p, ids, axis=-1)
    if normalize:
        w = w * _inverse(w.sum(axis=-1, keepdims=True))
    return ids, scale * w


def route_bwd(logits, ids, drw, score="softmax", normalize=True, scale=1.0):
    """Gradient of route's weights with respect to the logits, the choice held:
    dlogits [..., E] float64."""
    x = np.asarray(logits, np.float64)
    p = scores(x, score)
    q = np.take_along_axis(p, ids, axis=-1)
    g = scale * np.asarray(drw, np.float64)
    if normalize:
        inv = _inverse(q.sum(axis=-1, keepdims=True))
        g = (g - (g * q).sum(axis=-1, keepdims=True) * inv) * inv
    dp = np.zeros_like(p)
    np.put_along_axis(dp, ids, g, axis=-1)
    if score == "sigmoid":
        return dp * p * scores(-x, "sigmoid")
    return p * (dp - (dp * p).sum(axis=-1, keepdims=True))


def combine_bwd(plan, dout, y_nvs, rw_nvs):
    """dout [R,S,W] and y_nvs [R,NvS,W] bf16 bits, rw_nvs [R,NvS] fp32 ->
    (dy_nvs bits, drw [R,S,K] float64, bound [R,S,K]): the slots' gradients as
    bf16 of the fp32 product, zero where there is no token, and per route
    weight the sum of the products' magnitudes, which its rounding scales with."""
    R, S, K, NvS = plan.R, plan.S, plan.K, plan.NvS
    W = dout.shape[-1]
    slot = plan.dest.reshape(R * S, K)
    d = bf16_to_f32(dout.reshape(R * S, W))
    y = bf16_to_f32(y_nvs.reshape(R * NvS, W)).astype(np.float64)
    w = np.asarray(rw_nvs, np.float32).reshape(-1)
    dy = np.zeros((R * NvS, W), dtype=np.uint16)
    drw = np.zeros((R * S, K))
    bound = np.zeros((R * S, K))
    for k in range(K):
        dy[slot[:, k]] = f32_to_bf16((w[slot[:, k], None] * d).astype(np.float32))
        t = y[slot[:, k]] * d.astype(np.float64)
        drw[:, k] = t.sum(axis=1)
        bound[:, k] = np.abs(t).sum(axis=1)
    return dy.reshape(R, NvS, W), drw.reshape(R, S, K), bound.reshape(R, S, K)


def orthogonalize(g, coeffs, eps=1e-7):
    """Newton-Schulz iteration of one matrix in float64: X = G / (|G| + eps),
    then X = a X + (b A + c A A) X with A = X X^T for every (a, b, c)."""
    x = np.asarray(g, np.float64)
    x = x / (np.linalg.norm(x) + eps)
    if x.shape[0] > x.shape[1]:
        return orthogonalize_steps(x.T, coeffs).T
    return orthogonalize_steps(x, coeffs)


def orthogonalize_steps(x, coeffs):
    for a, b, c in coeffs:
        m = x @ x.T
        x = a * x + (b * m + c * (m @ m)) @ x
    return x
