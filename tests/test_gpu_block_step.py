"""A training step of one transformer block's expert half, as a framework runs
it: block_norm ends the block in front and norms for this one, router, plan,
dispatch, experts and combine beside shared_ffn, block_norm ends this block;
then all of their gradients.  Against a dense per-token computation in float64
that never sees a plan, against differences of its loss, and as a HIP graph
replayed for other tokens."""
import numpy as np
import pytest
import torch

import moonep_synth as synth
import oracle
from gpu_util import buffer_for, dev, dev_bf16, host_bf16, log, rel_l2
from grouped_gemm_moonep_amd import (block_norm, block_norm_bwd, block_norm_bwd_workspace,
                                     shared_ffn, shared_ffn_bwd, shared_ffn_bwd_workspace,
                                     shared_ffn_workspace)
from oracle import block as B
from oracle import swiglu
from oracle import training as T

pytestmark = pytest.mark.gpu

SHARED = 192                   # the shared expert's hidden size
SCALE1, SCALE2 = 1.0, 0.5
EPS = 1e-6
FORM = dict(score="sigmoid", normalize=True, scale=1.5)
# bf16 tensors that the step stores between the loss and its inputs: u, Z and Y of the routed and
# the shared experts, their sum, and on the way back dy, dY of the slots, dZ, dG, dU, dX of either, du
STORED = 12
f64 = lambda bits: oracle.bf16_to_f32(bits).astype(np.float64)


class Block:
    """Buffers of one step; every call writes the same tensors where the calls take them."""

    def __init__(self, w, home, joined):
        self.w, self.home, self.joined = w, home, joined
        self.buf = buffer_for(w)
        R, S, K, H, Hp, NvS = w.R, w.S, w.K, w.H, w.Hp, self.buf.NvS
        bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
        self.plan = self.buf.new_plan()
        self.pool = [bf(R, w.B, H, Hp) for _ in range(3)]
        self.x_nvs, self.y, self.dx_nvs, self.dy = (bf(R, NvS, H) for _ in range(4))
        self.z, self.dz, self.dg, self.du = (bf(R, NvS, Hp) for _ in range(4))
        self.ws = shared_ffn_workspace(R * S, H, SHARED)
        self.wsb = shared_ffn_bwd_workspace(R * S, H, SHARED)
        self.wsn = block_norm_bwd_workspace(R * S, H)

    def __call__(self, h, front, logits, p, dh2, du2):
        b, plan = self.buf, self.plan
        n1 = dict(gate=p["gate1"], w_post=p["post1"], w_pre=p["pre1"], scale=SCALE1, eps=EPS)
        n2 = dict(gate=p["gate2"], w_post=p["post2"], w_pre=p["pre2"], scale=SCALE2, eps=EPS)
        h1, u = block_norm(h, front, **n1)
        topk, rw = b.route(logits, **FORM)
        b.plan(topk, plan=plan)
        _, rw_nvs = b.dispatch(plan, u, rw, x_nvs=self.x_nvs)
        b.prefetch_weight(plan, self.home, self.pool)
        b.expert_ffn(plan, self.x_nvs, self.home, self.pool, z_ws=self.z, y_nvs=self.y)
        routed, _ = b.combine(plan, self.y, rw_nvs, gather_rw=False)
        if self.joined:
            outs = (shared_ffn(u, p["shared"], add=routed, ws=self.ws), None)
        else:
            outs = (routed, shared_ffn(u, p["shared"], ws=self.ws))
        h2, u2 = block_norm(h1, *outs, **n2)

        dh1, dy, dgate2, dpost2, dpre2 = block_norm_bwd(h2, dh2, du2, *outs, ws=self.wsn, **n2)
        du_s, dshared = shared_ffn_bwd(u, dy, p["shared"], ws=self.wsb)
        _, drw = b.combine_bwd(plan, dy, self.y, rw_nvs, dy_nvs=self.dy)
        b.expert_ffn_bwd(plan, self.x_nvs, self.dy, self.home, self.pool, self.dz, self.dg, self.du,
                         self.dx_nvs)
        du_r, _ = b.combine(plan, self.dx_nvs)
        dlogits = b.route_bwd(logits, topk, drw, **FORM)
        dh, dfront, dgate1, dpost1, dpre1 = block_norm_bwd(h1, dh1, du_s + du_r, front, ws=self.wsn,
                                                           **n1)
        return dict(h2=h2, u2=u2, topk=topk, h=dh, front=dfront, logits=dlogits, gate1=dgate1,
                    post1=dpost1, pre1=dpre1, gate2=dgate2, post2=dpost2, pre2=dpre2,
                    gate=dshared[0], up=dshared[1], down=dshared[2])


def case(dtype):
    w = synth.WORKLOADS["tiny_r4_s64_k2_e8"]
    home = [synth.expert_weights_host(w, i) for i in range(3)]
    home = [synth.to_bf16_bits(oracle.bf16_to_f32(t) * 4) for t in home]
    g = torch.Generator(device="cuda").manual_seed(11)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    R, S, H = w.R, w.S, w.H
    p = dict(gate1=torch.sigmoid(n(H)), post1=1 + 0.2 * n(H), pre1=1 + 0.2 * n(H),
             gate2=torch.sigmoid(n(R, S, 1)), post2=1 + 0.2 * n(H), pre2=1 + 0.2 * n(H),
             shared=tuple((n(H, SHARED) * s).bfloat16() for s in (0.13, 0.13, 0.07)))
    logits = n(R, S, w.E) - 0.3 * torch.arange(w.E, device="cuda")
    return (w, home, n(R, S, H).to(dtype), n(R, S, H).bfloat16(), logits, p,
            0.1 * n(R, S, H).to(dtype), (0.1 * n(R, S, H)).bfloat16())


@pytest.mark.parametrize("dtype,joined", [(torch.float32, False), (torch.bfloat16, True)])
def test_step_equals_dense_and_differences(dtype, joined):
    w, home, h, front, logits, p, dh2, du2 = case(dtype)
    log(f"block step {dtype} joined={joined}")
    step = Block(w, [dev_bf16(t) for t in home], joined)
    got = step(h, front, logits, p, dh2, du2)
    torch.cuda.synchronize()
    R, S, K, E, H = w.R, w.S, w.K, w.E, w.H
    ids = got["topk"].cpu().numpy()
    assert np.array_equal(ids, T.route(logits.cpu().numpy(), K, **FORM)[0])
    it = ids.reshape(R * S, K)
    num = lambda t: t.double().cpu().numpy()
    base = dict(h=num(h).reshape(-1, H), front=num(front).reshape(-1, H),
                logits=num(logits).reshape(-1, E), gate1=num(p["gate1"]), post1=num(p["post1"]),
                pre1=num(p["pre1"]), gate2=num(p["gate2"]).reshape(-1, 1), post2=num(p["post2"]),
                pre2=num(p["pre2"]), gate=num(p["shared"][0]), up=num(p["shared"][1]),
                down=num(p["shared"][2]))
    experts = [f64(t) for t in home]
    d1, d2 = num(dh2).reshape(-1, H), num(du2).reshape(-1, H)

    def forward(v):
        h1, u = B.block_norm(v["h"], v["front"], gate=v["gate1"], w_post=v["post1"],
                             w_pre=v["pre1"], scale=SCALE1, eps=EPS)
        q = np.take_along_axis(T.scores(v["logits"], "sigmoid"), it, -1)
        wt = 1.5 * q / q.sum(-1, keepdims=True)
        out = B.shared_ffn(u, (v["gate"], v["up"], v["down"]))
        for e in range(E):
            t, k = np.nonzero(it == e)
            if t.size:
                np.add.at(out, t, wt[t, k][:, None] * swiglu.forward(u[t], *(x[e] for x in experts))[1])
        return B.block_norm(h1, out, gate=v["gate2"], w_post=v["post2"], w_pre=v["pre2"],
                            scale=SCALE2, eps=EPS)

    h2, u2 = forward(base)
    assert rel_l2(num(got["h2"]).reshape(-1, H), h2) <= STORED / 2 * 2.0 ** -8
    assert rel_l2(num(got["u2"]).reshape(-1, H), u2) <= STORED / 2 * 2.0 ** -8

    def loss(v):
        a, c = forward(v)
        return float((d1 * a).sum() + (d2 * c).sum())

    rng = np.random.default_rng(3)
    for name, x in base.items():
        grad = num(got[name]).reshape(x.shape)
        for v in (grad / np.linalg.norm(grad), rng.standard_normal(x.shape)):
            s = 1e-4 / max(1.0, np.abs(v).max())
            fd = (loss({**base, name: x + s * v}) - loss({**base, name: x - s * v})) / (2 * s)
            tol = STORED * 2.0 ** -8 * np.linalg.norm(grad) * np.linalg.norm(v)
            assert abs((grad * v).sum() - fd) <= tol, name
    step.buf.destroy()


def test_step_graph_replays_equal_eager():
    w, home, h, front, logits, p, dh2, du2 = case(torch.bfloat16)
    step = Block(w, [dev_bf16(t) for t in home], False)
    ins = (h, front, logits, dh2, du2)
    perm = torch.randperm(w.S, generator=torch.Generator().manual_seed(1)).cuda()
    other = [[t.clone() for t in ins], [t[:, perm].contiguous() for t in ins],
             [t.flip(0).contiguous() for t in ins]]
    run = lambda a: step(a[0], a[1], a[2], p, a[3], a[4])
    refs = [{k: t.clone() for k, t in run(a).items()} for a in other]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(ins)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(ins)
    for rep in range(2):
        for a, ref in zip(other, refs):
            for t, v in zip(ins, a):
                t.copy_(v)
            for t in got.values():
                t.fill_(1)
            graph.replay()
            torch.cuda.synchronize()
            for k, t in got.items():
                assert torch.equal(t, ref[k]), k
            h.add_(0)
            torch.cuda.synchronize()
    del graph
    step.buf.destroy()


def test_decode_step():
    """One token per rank: the forward's calls at their smallest, against the same rows of a batch."""
    w, home, h, front, logits, p, _, _ = case(torch.bfloat16)
    n1 = dict(gate=p["gate1"], w_post=p["post1"], w_pre=p["pre1"], eps=EPS)
    h1, u = block_norm(h, front, **n1)
    s1, su = block_norm(h[:, :1].contiguous(), front[:, :1].contiguous(), **n1)
    assert torch.equal(h1[:, :1], s1) and torch.equal(u[:, :1], su)
    one, many = shared_ffn(su, p["shared"], add=s1), shared_ffn(u, p["shared"], add=h1)
    # the same products in another order of their sums
    a, b = one.double(), many[:, :1].double()
    assert (a - b).norm() <= 2.0 ** -8 * b.norm()
