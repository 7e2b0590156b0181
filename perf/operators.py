"""Measured cases of the training-step operators around the expert-parallel path.

Operators (the formulas are in include/moonep.h):

  route        the router's top-K choice and route weights from its logits
               (Buffer.route), what plan and dispatch take
  route_bwd    its gradient with respect to the logits (Buffer.route_bwd)
  combine_bwd  the gradient of the weighted combine with respect to the expert
               outputs and the route weights (Buffer.combine_bwd)
  ortho        the orthogonalised direction of a batch of weight gradients by
               Newton-Schulz products (orthogonalize)

`own` False: plain torch operations in 32 bits (the selection scores with a
bias in 64, since neighbours may differ by less than a rounding in 32).
`own` True: the framework's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
# the quintic Newton-Schulz coefficients of the Muon optimiser, five steps
COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of an 8-rank group, one token per rank: latency
        dict(name="route_decode", op="route", R=8, S=1, K=8, E=256, dtype="fp32",
             score="sigmoid", bias=True, normalize=True, scale=2.5),
        # a training microbatch of the README's Buffer example (fp32 logits)
        dict(name="route_train", op="route", R=8, S=4096, K=8, E=256, dtype="fp32",
             score="softmax", bias=False, normalize=True, scale=1.0),
        # the pages' benchmark shape, bias-balanced sigmoid scores, bf16 logits
        dict(name="route_pages", op="route", R=8, S=8192, K=8, E=384, dtype="bf16",
             score="sigmoid", bias=True, normalize=True, scale=2.5),
        # a ragged microbatch on the mid-size shape, probabilities as they are
        dict(name="route_ragged", op="route", R=8, S=1021, K=4, E=32, dtype="fp32",
             score="softmax", bias=False, normalize=False, scale=1.0),
        # the gradients of the second and of a ragged microbatch
        dict(name="route_bwd_train", op="route_bwd", R=8, S=4096, K=8, E=256, dtype="fp32",
             score="softmax", bias=False, normalize=True, scale=1.0),
        dict(name="route_bwd_ragged", op="route_bwd", R=8, S=2039, K=8, E=384, dtype="bf16",
             score="softmax", bias=False, normalize=False, scale=1.0),
        # the smallest workload, a ragged microbatch of the mid-size one and the
        # README's example (7168-wide rows of 262144 slots), Zipf-skewed routing
        dict(name="combine_bwd_tiny", op="combine_bwd", R=4, S=64, K=2, E=8, W=128, pad=16,
             zipf=0.5),
        dict(name="combine_bwd_ragged", op="combine_bwd", R=8, S=1021, K=4, E=32, W=1032, pad=128,
             zipf=0.3),
        dict(name="combine_bwd_train", op="combine_bwd", R=8, S=4096, K=8, E=256, W=7168, pad=128,
             zipf=0.5),
        # the gradients of every expert of the mid-size shape; of one rank's 32
        # home experts at the README's sizes; a few odd-sized bf16 momenta
        dict(name="ortho_mid", op="ortho", n=32, rows=1024, cols=2048, dtype="fp32"),
        dict(name="ortho_train", op="ortho", n=32, rows=7168, cols=2048, dtype="fp32"),
        dict(name="ortho_ragged", op="ortho", n=5, rows=509, cols=1283, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "combine_bwd", "ortho"])
    if op == "ortho":
        m, wide = _log_int(rng, 40, 2048), rng.uniform(1.0, 4.0)
        big = min(7168, int(m * wide))
        rows, cols = (m, big) if rng.random() < 0.5 else (big, m)
        most = 32 * 2048 * 2048 * (4 * 7168 + 2 * 2048) / (m * m * (4.0 * big + 2 * m))
        return dict(op=op, n=_log_int(rng, 1, max(1, min(32, int(most)))), rows=rows, cols=cols,
                    dtype=rng.choice(["fp32", "bf16"]))
    R = rng.choice([1, 2, 4, 8])
    E = R * rng.randint(max(1, 8 // R), 384 // R)
    K = rng.randint(1, min(8, E))
    if op == "combine_bwd":
        W = 8 * _log_int(rng, 8, 896)
        S = _log_int(rng, 1, max(1, min(4096, 8 * 4096 * 8 * 7168 // (R * K * W))))
        return dict(op=op, R=R, S=S, K=K, E=E, W=W, pad=rng.choice([1, 16, 128]),
                    zipf=rng.uniform(0.0, 1.0))
    normalize = rng.random() < 0.5
    if op == "route_bwd" and normalize:
        K = max(K, 2)               # the one weight of K = 1 is constant: no gradient
    return dict(op=op, R=R, S=_log_int(rng, 1, 8192 if op == "route" else 4096), K=K, E=E,
                dtype=rng.choice(["fp32", "bf16"]), score=rng.choice(["softmax", "sigmoid"]),
                bias=rng.random() < 0.5, normalize=normalize, scale=rng.choice([1.0, 2.5]))


def work(c):
    if c["op"] == "ortho":
        # the least arithmetic of the five steps known here: every step is a polynomial in the
        # Gram matrix, so one product of width max(rows, cols) at either end (the first one
        # symmetric) and 17 symmetric products of min(rows, cols)^2 between
        m, big = sorted((c["rows"], c["cols"]))
        size = 4 if c["dtype"] == "fp32" else 2
        gram = 3.0 * m * m * big + 17.0 * m ** 3
        steps = STEPS * (3.0 * m * m * big + m ** 3)
        return {"bytes": c["n"] * m * big * (size + 2), "flops": c["n"] * min(gram, steps)}
    T = c["R"] * c["S"]
    if c["op"] == "combine_bwd":
        return {"bytes": T * (2 * c["W"] * (1 + 2 * c["K"]) + 12 * c["K"]),
                "flops": 3.0 * T * c["K"] * c["W"]}
    size = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "route":
        return {"bytes": T * (size * c["E"] + 8 * c["K"]), "flops": 4.0 * T * c["E"]}
    dense = c["score"] == "softmax" and not c["normalize"]
    return {"bytes": T * (size * c["E"] + size * (c["E"] if dense else c["K"]) + 8 * c["K"]),
            "flops": T * (4.0 * c["E"] if dense else 8.0 * c["K"])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _logits(c, g):
    """Router logits of R S tokens: N(0, 1) times a few, with experts of unequal popularity."""
    x = torch.randn((c["R"], c["S"], c["E"]), generator=g, device=DEV)
    pop = torch.randn((c["E"],), generator=g, device=DEV)
    return (1.5 * x + 0.5 * pop).to(TYPES[c["dtype"]])


def _route_inputs(c, seed):
    g = _gen(seed)
    st = {"logits": _logits(c, g), "bias": None}
    if c["bias"]:
        st["bias"] = 0.05 * torch.randn((c["E"],), generator=g, device=DEV)
    return st, g


def _route_bwd_inputs(c, seed):
    st, g = _route_inputs(c, seed)
    key = st["logits"].double()
    if c["bias"]:
        key = (torch.softmax(key, -1) if c["score"] == "softmax" else torch.sigmoid(key)) + \
            st["bias"].double()
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    st["topk"] = order[..., :c["K"]].to(torch.int32).contiguous()
    st["drw"] = 0.1 * torch.randn(st["topk"].shape, generator=g, device=DEV)
    return st


def _layout(topk, E, pad):
    """Where the balanced plan puts every routed slot: (dest [R S K], padding slots, NvS).

    Each rank gets S K slots.  A group of experts above that gives to the ranks below it,
    the largest excess first; a donor short of a receiver's need gives it all the same and
    queues for the difference.  A group's experts lie on a line by (load, id) which its
    ranks cut into pieces; on a rank the home experts come first, then the others, each by
    id and rounded up to `pad` slots."""
    R, S, K = topk.shape
    L, C = E // R, S * K
    e_of = topk.reshape(-1).astype(np.int64)
    T = np.bincount(e_of, minlength=E)
    load = T.reshape(R, L).sum(1)
    keep, need = np.minimum(load, C), C - np.minimum(load, C)
    donors = sorted((g for g in range(R) if load[g] > C), key=lambda g: (C - load[g], g))
    queue = sorted((r for r in range(R) if need[r] > 0), key=lambda r: (-need[r], r))
    given, left = [[] for _ in range(R)], [int(load[g] - C) for g in donors]
    while queue:
        r, g = queue.pop(0), donors[0]
        given[g].append((int(need[r]), r))
        left[0] -= int(need[r])
        if left[0] < 0:
            keep[g] += left[0]
            need[g] = -left[0]
            queue.append(g)
        if left[0] <= 0 and len(donors) > 1:
            donors, left = donors[1:], left[1:]
    ends, ranks, at = [], [], 0
    for g in range(R):
        for n, r in [(int(keep[g]), g)] + given[g]:
            at += n
            ends.append(at)
            ranks.append(r)
    line = np.zeros(E, np.int64)            # expert -> start of its range, all groups in a row
    by = np.lexsort((np.arange(E), T, np.arange(E) // L))
    line[by] = np.cumsum(T[by]) - T[by]
    order = np.argsort(e_of, kind="stable")
    e = e_of[order]
    pos = line[e] + np.arange(e.size) - (np.cumsum(T) - T)[e]
    d = np.asarray(ranks)[np.searchsorted(np.asarray(ends), pos, side="right")]
    seg = d * 2 * E + np.where(e // L == d, e, E + e)
    segs, inv, cnt = np.unique(seg, return_inverse=True, return_counts=True)
    length = -(-cnt // pad) * pad
    start = np.cumsum(length) - length
    rank = segs // (2 * E)
    start -= start[np.searchsorted(rank, rank)]          # from the rank's first slot
    nvs = C + 2 * L * pad
    first = rank * nvs + start
    o = np.argsort(inv, kind="stable")
    within = np.empty(e.size, np.int64)
    within[o] = np.arange(e.size) - np.repeat(np.cumsum(cnt) - cnt, cnt)
    dest = np.empty(e.size, np.int64)
    dest[order] = first[inv] + within
    gap = length - cnt
    padding = np.repeat(first + cnt - (np.cumsum(gap) - gap), gap) + np.arange(gap.sum())
    return dest, padding, nvs


def _combine_inputs(c, seed):
    """A routed microbatch with Zipf-popular experts, its expert outputs and output gradient."""
    g = _gen(seed)
    R, S, K, E, W = c["R"], c["S"], c["K"], c["E"], c["W"]
    score = torch.randn((R, S, E), generator=g, device=DEV) - \
        c["zipf"] * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    top = torch.topk(score, K, dim=-1)
    topk = top.indices.to(torch.int32).contiguous()
    dest, padding, nvs = _layout(topk.cpu().numpy(), E, c["pad"])
    dest, padding = torch.from_numpy(dest).to(DEV), torch.from_numpy(padding).to(DEV)
    rw_nvs = torch.zeros((R, nvs), device=DEV)
    rw_nvs.view(-1)[dest] = torch.softmax(top.values, -1).reshape(-1)
    y = torch.empty((R, nvs, W), dtype=torch.bfloat16, device=DEV)
    for r in range(R):
        y[r] = torch.randn((nvs, W), generator=g, device=DEV)
    y.view(-1, W)[padding] = 0
    dout = (0.01 * torch.randn((R, S, W), generator=g, device=DEV)).to(torch.bfloat16)
    return {"topk": topk, "dest": dest, "padding": padding, "y": y, "rw_nvs": rw_nvs, "dout": dout}


def _ortho_inputs(c, seed):
    """Weight gradients A^T B of segments of unequal length: one of few tokens has a low rank,
    one of none is zero."""
    g = _gen(seed)
    n, rows, cols = c["n"], c["rows"], c["cols"]
    out = torch.empty((n, rows, cols), dtype=TYPES[c["dtype"]], device=DEV)
    tok = (torch.rand((n,), generator=g, device=DEV) * math.log(2.0 * min(rows, cols))).exp()
    scale = torch.exp(torch.randn((rows,), generator=g, device=DEV))
    for i, t in enumerate(tok.long().tolist()):
        t = 0 if n >= 8 and i == 1 else max(t, 1)
        a = torch.randn((t, rows), generator=g, device=DEV) * scale
        b = 1e-3 * torch.randn((t, cols), generator=g, device=DEV)
        out[i] = a.t() @ b
    return out


def prepare(case, seed):
    op = case["op"]
    if op == "ortho":
        st = {"g": _ortho_inputs(case, seed)}
    elif op == "route":
        st = _route_inputs(case, seed)[0]
    elif op == "route_bwd":
        st = _route_bwd_inputs(case, seed)
    else:
        st = _combine_inputs(case, seed)
        # the slots behind a rank's last segment keep what they hold
        st["dy"] = torch.zeros_like(st["y"])
    st["case"] = case
    if own:
        # the handle, the microbatch's plan and the workspace, which a training program holds
        import grouped_gemm_moonep_amd as moonep
        st["moonep"] = moonep
        if op == "ortho":
            st["ws"] = moonep.orthogonalize_workspace(*st["g"].shape)
        else:
            W = case.get("W", 64)
            st["buf"] = moonep.Buffer(R=case["R"], S=case["S"], K=case["K"], E=case["E"],
                                      H=(W + 63) // 64 * 64, Hp=64,
                                      token_padding=case.get("pad", 128))
            if op == "combine_bwd":
                st["plan"] = st["buf"].plan(st["topk"])
    return st


# ------------------------------------------------------------- plain forms
def _plain_scores(x, score):
    """Scores of the logits; a token with no open expert has scores of zero."""
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    s = e.sum(-1, keepdim=True)
    return e / torch.where(s == 0, torch.ones_like(s), s)


def _plain_route(c, st):
    x = st["logits"].float()
    if st["bias"] is None:
        key = x
    else:
        key = _plain_scores(x.double(), c["score"]) + st["bias"].double()
        key = torch.where(x == -math.inf, x.double(), key)
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :c["K"]]
    if c["score"] == "softmax" and c["normalize"]:
        w = _plain_scores(x.gather(-1, ids), "softmax")
    else:
        w = _plain_scores(x, c["score"]).gather(-1, ids)
        if c["normalize"]:
            s = w.sum(-1, keepdim=True)
            w = w / torch.where(s == 0, torch.ones_like(s), s)
    return ids.to(torch.int32), w * c["scale"]


def _plain_route_bwd(c, st):
    x, ids, dw = st["logits"].float(), st["topk"].long(), st["drw"] * c["scale"]
    if c["score"] == "softmax" and c["normalize"]:
        w = _plain_scores(x.gather(-1, ids), "softmax")
        d = w * (dw - (dw * w).sum(-1, keepdim=True))
        return torch.zeros_like(x).scatter_(-1, ids, d).to(st["logits"].dtype)
    s = _plain_scores(x, c["score"])
    p = s.gather(-1, ids)
    if c["score"] == "softmax":
        d = -s * (dw * p).sum(-1, keepdim=True)
        return d.scatter_add_(-1, ids, dw * p).to(st["logits"].dtype)
    if c["normalize"]:
        total = p.sum(-1, keepdim=True)
        total = torch.where(total == 0, torch.ones_like(total), total)
        dw = (dw - (dw * p).sum(-1, keepdim=True) / total) / total
    return torch.zeros_like(x).scatter_(-1, ids, dw * p * (1.0 - p)).to(st["logits"].dtype)


def _plain_combine_bwd(c, st):
    W, K = c["W"], c["K"]
    dest = st["dest"]
    d = st["dout"].reshape(-1, 1, W).float()
    w = st["rw_nvs"].reshape(-1)[dest].reshape(-1, K, 1)
    drw = (st["y"].reshape(-1, W)[dest].reshape(-1, K, W).float() * d).sum(-1)
    dy = st["dy"]
    dy.view(-1, W)[dest] = (w * d).to(torch.bfloat16).reshape(-1, W)
    dy.view(-1, W)[st["padding"]] = 0
    return dy, drw.reshape(c["R"], c["S"], K)


def _plain_step(x):
    a, b, c = COEFFS
    s = x @ x.transpose(1, 2)
    return a * x + (b * s + c * (s @ s)) @ x


def _plain_ortho(g):
    x = g.float()
    norm = (x.double() * x.double()).sum((1, 2), keepdim=True).sqrt()
    x = x * (1.0 / (norm + EPS)).float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    for _ in range(STEPS):
        x = _plain_step(x)
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous()


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        if op == "ortho":
            return state["moonep"].orthogonalize(state["g"], steps=STEPS, coeffs=COEFFS, eps=EPS,
                                                 ws=state["ws"])
        buf = state["buf"]
        if op == "combine_bwd":
            return buf.combine_bwd(state["plan"], state["dout"], state["y"], state["rw_nvs"],
                                   dy_nvs=state["dy"])
        form = dict(score=c["score"], normalize=c["normalize"], scale=c["scale"])
        if op == "route":
            return buf.route(state["logits"], state["bias"], **form)
        return buf.route_bwd(state["logits"], state["topk"], state["drw"], **form)
    if op == "ortho":
        return _plain_ortho(state["g"])
    if op == "combine_bwd":
        return _plain_combine_bwd(c, state)
    return _plain_route(c, state) if op == "route" else _plain_route_bwd(c, state)


# ------------------------------------------------------ 64-bit definitions
def _exact_prob(x, score):
    """x: numpy float64 [tokens, E]."""
    if score == "sigmoid":
        return 1.0 / (1.0 + np.exp(-x))
    e = np.exp(x - x.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True)


def _exact_route(c, seed):
    st = _route_inputs(c, seed)[0]
    x = st["logits"].double().cpu().numpy().reshape(-1, c["E"])
    p = _exact_prob(x, c["score"])
    rank = x if st["bias"] is None else p + st["bias"].double().cpu().numpy()
    ids = np.argsort(-rank, axis=1, kind="stable")[:, :c["K"]]
    w = np.take_along_axis(p, ids, axis=1)
    if c["normalize"]:
        w /= w.sum(axis=1, keepdims=True)
    shape = (c["R"], c["S"], c["K"])
    return ids.astype(np.int32).reshape(shape), (c["scale"] * w).reshape(shape)


def _exact_route_bwd(c, seed):
    st = _route_bwd_inputs(c, seed)
    x = st["logits"].double().cpu().numpy().reshape(-1, c["E"])
    ids = st["topk"].cpu().numpy().reshape(-1, c["K"]).astype(np.int64)
    dw = st["drw"].double().cpu().numpy().reshape(-1, c["K"])
    p = _exact_prob(x, c["score"])
    q = np.take_along_axis(p, ids, axis=1)
    # through w = scale q / sum(q), or w = scale q
    if c["normalize"]:
        t = q.sum(axis=1, keepdims=True)
        dq = c["scale"] * (dw / t - (dw * q).sum(axis=1, keepdims=True) / t ** 2)
    else:
        dq = c["scale"] * dw
    dp = np.zeros_like(p)
    np.put_along_axis(dp, ids, dq, axis=1)
    # through the score function
    if c["score"] == "sigmoid":
        dx = dp * p * (1.0 - p)
    else:
        dx = p * (dp - (dp * p).sum(axis=1, keepdims=True))
    return dx.reshape(c["R"], c["S"], c["E"])


def _exact_combine_bwd(c, seed):
    st = _combine_inputs(c, seed)
    T, K, W = c["R"] * c["S"], c["K"], c["W"]
    slot = st["dest"].reshape(T, K)
    y, w = st["y"].reshape(-1, W), st["rw_nvs"].reshape(-1).double()
    dy = torch.zeros(y.shape, dtype=torch.float64, device=y.device)
    drw = torch.empty((T, K), dtype=torch.float64, device=y.device)
    for t0 in range(0, T, 4096):
        d = st["dout"].reshape(T, W)[t0:t0 + 4096].double()
        for k in range(K):
            s = slot[t0:t0 + 4096, k]
            drw[t0:t0 + 4096, k] = torch.linalg.vecdot(d, y[s].double())
            dy.index_copy_(0, s, w[s, None] * d)
    return dy.reshape(st["y"].shape), drw.reshape(c["R"], c["S"], K)


def _exact_ortho(c, seed):
    g = _ortho_inputs(c, seed)
    a, b, e = COEFFS
    out = torch.empty(g.shape, dtype=torch.float64, device=g.device)
    for i in range(g.shape[0]):
        x = g[i].double()
        x = x / (torch.linalg.matrix_norm(x) + EPS)
        short = x.shape[0] <= x.shape[1]
        for _ in range(STEPS):
            gram = x.mm(x.t()) if short else x.t().mm(x)
            q = torch.addmm(b * gram, gram, gram, alpha=e)
            q.diagonal().add_(a)
            x = q.mm(x) if short else x.mm(q)
        out[i] = x
    return out


def exact(case, seed):
    return {"route": _exact_route, "route_bwd": _exact_route_bwd,
            "combine_bwd": _exact_combine_bwd, "ortho": _exact_ortho}[case["op"]](case, seed)
