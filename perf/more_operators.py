"""Measured cases of the operators that surround the expert path inside one transformer block.

Operators (the formulas are in include/moonep.h):

  norm       a block's end and the next one's start in one pass: the block's outputs are
             summed, normalised, gated, scaled and added to the residual stream, and the
             stream is normalised for what comes next (block_norm)
  norm_bwd   its gradients: stream, block output, gate and both norms' weights (block_norm_bwd)
  ffn        the shared expert, a gated feed-forward block of every token, added to the
             routed experts' combined output (shared_ffn)
  ffn_bwd    its gradients: tokens and the three projections (shared_ffn_bwd)

`own` False: plain torch operations in 32 bits, rounded once at the end.
`own` True: the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
GATES = ("none", "channel", "token", "full")


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of an 8-rank group, one token per rank: latency
        dict(name="norm_decode", op="norm", T=8, W=7168, dtype="bf16", two=True, gate="none",
             post=False, pre=True, scale=1.0),
        # a training microbatch of the README's Buffer example: routed and shared experts'
        # outputs, norms on both sides of the block, a learned gate per channel
        dict(name="norm_train", op="norm", T=32768, W=7168, dtype="bf16", two=True,
             gate="channel", post=True, pre=True, scale=0.5),
        # a ragged microbatch of rows that are no multiple of a wave, stream in fp32,
        # a gate per token
        dict(name="norm_ragged", op="norm", T=8168, W=1032, dtype="fp32", two=False,
             gate="token", post=True, pre=True, scale=1.0),
        # their gradients: the smallest workload's tokens, the training microbatch, and the
        # ragged one with a gate of its own for every element
        dict(name="norm_bwd_tiny", op="norm_bwd", T=256, W=128, dtype="bf16", two=False,
             gate="channel", post=True, pre=True, scale=1.0),
        dict(name="norm_bwd_train", op="norm_bwd", T=32768, W=7168, dtype="bf16", two=True,
             gate="channel", post=True, pre=True, scale=0.5),
        dict(name="norm_bwd_ragged", op="norm_bwd", T=8168, W=1032, dtype="fp32", two=False,
             gate="full", post=True, pre=True, scale=1.0),
        # the shared expert in one decode step, in the inference workload's step of 8 x 128
        # tokens, in a ragged microbatch of the mid-size shape, in the training microbatch
        dict(name="ffn_decode", op="ffn", T=8, H=7168, Hp=2048, act="silu", add=True),
        dict(name="ffn_infer", op="ffn", T=1024, H=7168, Hp=2048, act="silu", add=True),
        dict(name="ffn_ragged", op="ffn", T=8168, H=1024, Hp=2048, act="gelu_tanh", add=False),
        dict(name="ffn_train", op="ffn", T=32768, H=7168, Hp=2048, act="silu", add=True),
        # its gradients: the smallest workload and the training microbatch
        dict(name="ffn_bwd_tiny", op="ffn_bwd", T=256, H=128, Hp=256, act="gelu_tanh"),
        dict(name="ffn_bwd_train", op="ffn_bwd", T=32768, H=7168, Hp=2048, act="silu"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "ffn", "ffn_bwd"])
    if op in ("ffn", "ffn_bwd"):
        H = 64 * _log_int(rng, 2, 112)
        Hp = 64 * _log_int(rng, 1, 64)
        T = _log_int(rng, 1, min(32768, 32768 * 7168 * 2048 // (H * Hp)))
        c = dict(op=op, T=T, H=H, Hp=Hp, act=rng.choice(["silu", "gelu_tanh"]))
        if op == "ffn":
            c["add"] = rng.random() < 0.5
        return c
    dtype = rng.choice(["fp32", "bf16"])
    W = 8 * _log_int(rng, 8, 896)
    # an fp32 stream and a full gate move up to twice the bytes
    T = _log_int(rng, 1, 16384 if dtype == "fp32" else 32768)
    post = rng.random() < 0.7
    return dict(op=op, T=T, W=W, dtype=dtype, two=rng.random() < 0.5,
                gate=rng.choice(GATES if T <= 16384 else GATES[:3]), post=post,
                pre=not post or rng.random() < 0.8, scale=rng.choice([1.0, 0.5, 0.22]))


def work(c):
    T = c["T"]
    if c["op"] == "ffn":
        return {"bytes": 2 * (T * c["H"] * (3 if c["add"] else 2) + 3 * c["H"] * c["Hp"]),
                "flops": 6.0 * T * c["H"] * c["Hp"]}
    if c["op"] == "ffn_bwd":
        # gate and up again, dZ, dX (two products) and the three weight gradients
        return {"bytes": 2 * (T * c["H"] * 3 + 6 * c["H"] * c["Hp"]),
                "flops": 16.0 * T * c["H"] * c["Hp"]}
    n = T * c["W"]
    stream = 4 if c["dtype"] == "fp32" else 2
    gate = {"none": 0, "channel": 4 * c["W"], "token": 4 * T, "full": 2 * n}[c["gate"]]
    weights = 4 * c["W"] * (c["post"] + c["pre"])
    outs = 2 * n * (2 if c["two"] else 1)
    if c["op"] == "norm":
        return {"bytes": n * (2 * stream + 2 * c["pre"]) + outs + gate + weights,
                "flops": n * (3.0 + 3 * c["post"] + 3 * c["pre"])}
    # stream, its gradient, du in; block outputs in where the norm or the gate needs them
    need = c["post"] or c["gate"] != "none"
    return {"bytes": n * (2 * stream + 2) + (n * (stream + 2) if c["pre"] else 0) +
            (outs if need else 0) + 2 * gate + 2 * weights,
            "flops": n * (2.0 + 8 * c["post"] + 8 * c["pre"])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ffn_inputs(c, seed):
    """Normalised tokens; projections that keep the activations around one."""
    g = _gen(seed)
    T, H, Hp = c["T"], c["H"], c["Hp"]

    def bf(shape, sd):
        return torch.empty(shape, device=DEV).normal_(0.0, sd, generator=g).to(torch.bfloat16)

    st = {"x": bf((T, H), 1.0),
          "w": (bf((H, Hp), 1.5 / math.sqrt(H)), bf((H, Hp), 1.5 / math.sqrt(H)),
                bf((H, Hp), 1.0 / math.sqrt(Hp)))}
    if c["op"] == "ffn_bwd":
        st["dy"] = bf((T, H), 0.01)
    else:
        st["add"] = bf((T, H), 1.0) if c["add"] else None
    return st


def _norm_inputs(c, seed):
    """A residual stream with a few large channels, block outputs whose size differs from token
    to token, weights around one, gates between zero and one."""
    g = _gen(seed)
    T, W = c["T"], c["W"]

    def nrm(*shape):
        return torch.empty(shape, device=DEV).normal_(generator=g)

    st = {"y2": None, "gate": None, "w_post": None, "w_pre": None}
    chan = torch.exp(0.7 * nrm(W))
    st["h"] = (nrm(T, W) * chan).to(TYPES[c["dtype"]])
    size = torch.exp(nrm(T, 1))
    st["y"] = (nrm(T, W) * size).to(torch.bfloat16)
    if c["two"]:
        st["y2"] = (0.5 * nrm(T, W)).to(torch.bfloat16)
    if c["gate"] == "channel":
        st["gate"] = torch.sigmoid(nrm(W))
    elif c["gate"] == "token":
        st["gate"] = torch.sigmoid(nrm(T, 1))
    elif c["gate"] == "full":
        st["gate"] = torch.sigmoid(nrm(T, W)).to(torch.bfloat16)
    if c["post"]:
        st["w_post"] = 1.0 + 0.2 * nrm(W)
    if c["pre"]:
        st["w_pre"] = 1.0 + 0.2 * nrm(W)
    if c["op"] == "norm_bwd":
        st["dh"] = (0.01 * nrm(T, W)).to(TYPES[c["dtype"]])
        st["du"] = (0.01 * nrm(T, W)).to(torch.bfloat16) if c["pre"] else None
    return st


def prepare(case, seed):
    op = case["op"]
    st = _ffn_inputs(case, seed) if op in ("ffn", "ffn_bwd") else _norm_inputs(case, seed)
    st["case"] = case
    if own:
        # the workspace, which a program keeps
        import grouped_gemm_moonep_amd as moonep
        st["moonep"] = moonep
        if op in ("ffn", "ffn_bwd"):
            make = (moonep.shared_ffn_workspace if op == "ffn" else
                    moonep.shared_ffn_bwd_workspace)
            st["ws"] = make(case["T"], case["H"], case["Hp"])
        elif op == "norm_bwd":
            st["ws"] = moonep.block_norm_bwd_workspace(case["T"], case["W"])
    return st


# ------------------------------------------------------------- plain forms
def _plain_act(act, g):
    """(activation, derivative) of g sigma(c(g))."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    k = 2.0 * math.sqrt(2.0 / math.pi)
    s = 1.0 / (1.0 + torch.exp(-k * (g + 0.044715 * g * g * g)))
    return g * s, s * (1.0 + g * (1.0 - s) * k * (1.0 + 3 * 0.044715 * g * g))


def _plain_ffn(c, st):
    x, (wg, wu, wd) = st["x"].float(), (w.float() for w in st["w"])
    a, _ = _plain_act(c["act"], x @ wg)
    y = (a * (x @ wu)) @ wd.t()
    if st["add"] is not None:
        y = y + st["add"].float()
    return y.to(torch.bfloat16)


def _plain_ffn_bwd(c, st):
    x, dy, (wg, wu, wd) = st["x"].float(), st["dy"].float(), (w.float() for w in st["w"])
    a, da = _plain_act(c["act"], x @ wg)
    u = x @ wu
    dz = dy @ wd
    dg, du = dz * u * da, dz * a
    dx = dg @ wg.t() + du @ wu.t()
    return tuple(t.to(torch.bfloat16) for t in (dx, x.t() @ dg, x.t() @ du, dy.t() @ (a * u)))


def _rstd(v):
    return 1.0 / torch.sqrt((v * v).sum(-1, keepdim=True) / v.shape[-1] + EPS)


def _plain_block(st):
    a = st["y"].float()
    return a if st["y2"] is None else a + st["y2"].float()


def _plain_norm(c, st):
    n = _plain_block(st)
    if st["w_post"] is not None:
        n = n * _rstd(n) * st["w_post"]
    if st["gate"] is not None:
        n = n * st["gate"].float()
    h = st["h"].float() + c["scale"] * n
    u = None
    if st["w_pre"] is not None:
        u = (h * _rstd(h) * st["w_pre"]).to(torch.bfloat16)
    return h.to(st["h"].dtype), u


def _plain_norm_bwd(c, st):
    d, dw_pre, dgate, dw_post = st["dh"].float(), None, None, None
    W = c["W"]
    if st["du"] is not None:
        h, du = st["h"].float(), st["du"].float()
        r = _rstd(h)
        hat, v = h * r, du * st["w_pre"]
        dw_pre = (du * hat).sum(0)
        d = d + r * (v - hat * ((v * hat).sum(-1, keepdim=True) / W))
    a = _plain_block(st)
    r = _rstd(a)
    n = a if st["w_post"] is None else a * r * st["w_post"]
    dn = c["scale"] * d
    if st["gate"] is not None:
        t = dn * n
        dgate = {"channel": lambda: t.sum(0), "token": lambda: t.sum(-1, keepdim=True),
                 "full": lambda: t.to(torch.bfloat16)}[c["gate"]]()
        dn = dn * st["gate"].float()
    if st["w_post"] is not None:
        hat = a * r
        dw_post = (dn * hat).sum(0)
        v = dn * st["w_post"]
        dn = r * (v - hat * ((v * hat).sum(-1, keepdim=True) / W))
    return d.to(st["dh"].dtype), dn.to(torch.bfloat16), dgate, dw_post, dw_pre


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        m = state["moonep"]
        if op == "ffn":
            return m.shared_ffn(state["x"], state["w"], act=c["act"], add=state["add"],
                                ws=state["ws"])
        if op == "ffn_bwd":
            dx, dw = m.shared_ffn_bwd(state["x"], state["dy"], state["w"], act=c["act"],
                                      ws=state["ws"])
            return dx, dw[0], dw[1], dw[2]
        form = dict(gate=state["gate"], w_post=state["w_post"], w_pre=state["w_pre"],
                    scale=c["scale"], eps=EPS)
        if op == "norm":
            return m.block_norm(state["h"], state["y"], state["y2"], **form)
        return m.block_norm_bwd(state["h"], state["dh"], state["du"], state["y"], state["y2"],
                                ws=state["ws"], **form)
    return {"ffn": _plain_ffn, "ffn_bwd": _plain_ffn_bwd, "norm": _plain_norm,
            "norm_bwd": _plain_norm_bwd}[op](c, state)


# ------------------------------------------------------ 64-bit definitions
def _def_ffn(c, x, wg, wu, wd):
    g = torch.mm(x, wg)
    if c["act"] == "silu":
        a = torch.nn.functional.silu(g)
    else:
        inner = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g.pow(3))
        a = 0.5 * g * (1.0 + torch.tanh(inner))
    return torch.mm(a * torch.mm(x, wu), wd.t())


def _def_norm(c, h, y, y2, gate, w_post, w_pre):
    def rms(v, w):
        return w * v / (v.square().mean(-1, keepdim=True) + EPS).sqrt()

    n = y if y2 is None else y + y2
    n = n if w_post is None else rms(n, w_post)
    n = n if gate is None else gate * n
    out = torch.add(h, n, alpha=c["scale"])
    return out, None if w_pre is None else rms(out, w_pre)


def _wide(t):
    return None if t is None else t.double()


def exact(case, seed):
    c = case
    if c["op"] == "ffn":
        st = _ffn_inputs(c, seed)
        w = [t.double() for t in st["w"]]
        y = torch.cat([_def_ffn(c, x.double(), *w) for x in st["x"].split(8192)])
        return y if st["add"] is None else y.add_(st["add"])
    if c["op"] == "ffn_bwd":
        st = _ffn_inputs(c, seed)
        w = [t.double().requires_grad_() for t in st["w"]]
        dx = []
        for x, dy in zip(st["x"].split(8192), st["dy"].split(8192)):
            x = x.double().requires_grad_()
            _def_ffn(c, x, *w).backward(dy.double())
            dx.append(x.grad)
        return (torch.cat(dx), *(t.grad for t in w))
    st = _norm_inputs(c, seed)
    names = ("y", "y2", "gate", "w_post", "w_pre")
    if c["op"] == "norm":
        return _def_norm(c, st["h"].double(), *(_wide(st[n]) for n in names))
    # the gradients of <dh, out> + <du, rms(out)> at a stream whose sum is the given one
    v = {n: None if st[n] is None else st[n].double().requires_grad_() for n in names}
    add = _def_norm(c, torch.zeros_like(st["h"], dtype=torch.float64),
                    v["y"], v["y2"], v["gate"], v["w_post"], None)[0]
    before = (st["h"].double() - add.detach()).requires_grad_()
    out = before + add
    u = None if v["w_pre"] is None else _def_norm(dict(c, scale=0.0), out, torch.zeros_like(out),
                                                  None, None, None, v["w_pre"])[1]
    roots, grads = [out], [st["dh"].double()]
    if u is not None:
        roots.append(u)
        grads.append(st["du"].double())
    torch.autograd.backward(roots, grads)
    got = [None if v[n] is None else v[n].grad for n in ("gate", "w_post", "w_pre")]
    return (before.grad, v["y"].grad, *got)
