"""A training step of the whole MoE layer with route weights in the combine,
from router logits to update directions: route, plan, dispatch, prefetch, FFN,
weighted combine; combine_bwd, FFN backward, dispatch bwd, weight gradients,
reduce_grad, route_bwd, orthogonalize.  Against a dense per-token computation
in float64 that never sees a plan, against differences of its loss, and as a
HIP graph replayed for other tokens."""
import numpy as np
import pytest
import torch

import moonep_synth as synth
import oracle
from gpu_util import assert_close_bf16, buffer_for, dev, dev_bf16, host_bf16, log, rel_l2
from grouped_gemm_moonep_amd import MUON_COEFFS, orthogonalize, orthogonalize_workspace
from oracle import swiglu
from oracle import training as T

pytestmark = pytest.mark.gpu

f64 = lambda bits: oracle.bf16_to_f32(bits).astype(np.float64)


class Step:
    """Buffers of one step; every call writes the same tensors."""

    def __init__(self, w, home, **form):
        self.w, self.home, self.form = w, home, form
        self.buf = buffer_for(w)
        R, S, K, E, H, Hp, NvS = w.R, w.S, w.K, w.E, w.H, w.Hp, self.buf.NvS
        bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
        f32 = lambda *s: torch.zeros(s, dtype=torch.float32, device="cuda")
        self.plan = self.buf.new_plan()
        self.pool = [bf(R, w.B, H, Hp) for _ in range(3)]
        self.topk = torch.zeros((R, S, K), dtype=torch.int32, device="cuda")
        self.rw, self.drw, self.rw_nvs = f32(R, S, K), f32(R, S, K), f32(R, NvS)
        self.x_nvs, self.y, self.dx_nvs = bf(R, NvS, H), bf(R, NvS, H), bf(R, NvS, H)
        self.z, self.dz, self.dg, self.du = (bf(R, NvS, Hp) for _ in range(4))
        self.dy = bf(R, NvS, H)
        self.out, self.dx = bf(R, S, H), bf(R, S, H)
        self.dlogits = f32(R, S, E)
        self.grads = [f32(E, H, Hp) for _ in range(3)]
        self.rbuf = [f32(R, w.B, H, Hp) for _ in range(3)]
        self.ws = orthogonalize_workspace(E, H, Hp)
        self.dirs = [bf(E, H, Hp) for _ in range(3)]

    def __call__(self, x, logits, dout):
        b, p = self.buf, self.plan
        b.route(logits, topk=self.topk, rw=self.rw, **self.form)
        b.plan(self.topk, plan=p)
        b.dispatch(p, x, self.rw, x_nvs=self.x_nvs, rw_nvs=self.rw_nvs)
        b.prefetch_weight(p, self.home, self.pool)
        b.expert_ffn(p, self.x_nvs, self.home, self.pool, z_ws=self.z, y_nvs=self.y)
        b.combine(p, self.y, self.rw_nvs, out=self.out, gather_rw=False)
        b.combine_bwd(p, dout, self.y, self.rw_nvs, dy_nvs=self.dy, drw=self.drw)
        b.expert_ffn_bwd(p, self.x_nvs, self.dy, self.home, self.pool, self.dz, self.dg, self.du,
                         self.dx_nvs)
        b.combine(p, self.dx_nvs, out=self.dx)
        for g in self.grads:
            g.zero_()
        for i, (a, c) in enumerate(((self.x_nvs, self.dg), (self.x_nvs, self.du), (self.dy, self.z))):
            b.expert_wgrad(p, a, c, self.grads[i], self.rbuf[i])
        b.reduce_grad(p, self.grads, self.rbuf)
        b.route_bwd(logits, self.topk, self.drw, dlogits=self.dlogits, **self.form)
        for g, d in zip(self.grads, self.dirs):
            orthogonalize(g, out=d, ws=self.ws)

    def results(self):
        return [self.topk, self.rw, self.out, self.dx, self.dlogits, *self.grads, *self.dirs]


def case(score):
    w = synth.WORKLOADS["tiny_r4_s64_k2_e8"]
    home_h = [synth.expert_weights_host(w, i) for i in range(3)]
    home_h = [synth.to_bf16_bits(oracle.bf16_to_f32(h) * 4) for h in home_h]   # outputs near one
    logits = synth.rng(0, 17).standard_normal((w.R, w.S, w.E), dtype=np.float32)
    logits -= (0.3 * np.arange(w.E)).astype(np.float32)
    form = dict(score=score, normalize=True, scale=1.5)
    return w, home_h, synth.hidden(w), logits, synth.grad_out(w, w.H), form


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_step_equals_dense_and_differences(score):
    w, home_h, x, logits, dout, form = case(score)
    log(f"weighted step {score}")
    step = Step(w, [dev_bf16(h) for h in home_h], **form)
    step(dev_bf16(x), dev(logits), dev_bf16(dout))
    torch.cuda.synchronize()
    R, S, K, E, H = w.R, w.S, w.K, w.E, w.H
    ids, rw = T.route(logits, K, **form)
    assert np.array_equal(step.topk.cpu().numpy(), ids)
    rw32 = step.rw.cpu().numpy()

    # dense, token-major, rounded where the path stores bf16
    xt, dt, it = x.reshape(R * S, H), dout.reshape(R * S, H), ids.reshape(R * S, K)
    wt = rw32.reshape(R * S, K)
    y = np.zeros((R * S, K, H), np.uint16)
    dx_k = np.zeros_like(y)
    drw = np.zeros((R * S, K))
    gw = [np.zeros((E, H, w.Hp)) for _ in range(3)]
    for e in range(E):
        t, k = np.nonzero(it == e)
        if not t.size:
            continue
        z_e, y_e = oracle.ffn_token(xt[t], *(h[e] for h in home_h))
        y[t, k] = y_e
        drw[t, k] = (f64(y_e) * f64(dt[t])).sum(1)
        dy_e = oracle.f32_to_bf16((wt[t, k][:, None] * oracle.bf16_to_f32(dt[t])).astype(np.float32))
        _, dg, du, dx_e = oracle.ffn_token_backward(xt[t], dy_e, *(h[e] for h in home_h))
        dx_k[t, k] = dx_e
        gw[0][e], gw[1][e] = f64(xt[t]).T @ f64(dg), f64(xt[t]).T @ f64(du)
        gw[2][e] = f64(dy_e).T @ f64(z_e)
    assert_close_bf16(host_bf16(step.out),
                      oracle.combine_rows(y, wt).reshape(R, S, H), what="out")
    assert_close_bf16(host_bf16(step.dx), oracle.combine_rows(dx_k).reshape(R, S, H), what="dx",
                      ulps=2)
    # y differs by a rounding here and there: 2^-8 of a few of the terms of each sum
    assert rel_l2(step.drw.cpu().numpy().reshape(R * S, K), drw) < 2.0 ** -8
    dl = T.route_bwd(logits, ids, drw.reshape(R, S, K), **form)
    got_dl = step.dlogits.cpu().numpy().astype(np.float64)
    assert rel_l2(got_dl, dl) < 2.0 ** -7
    for i, nm in enumerate(("dWg", "dWu", "dWd")):
        got = step.grads[i].cpu().numpy().astype(np.float64)
        assert rel_l2(got, gw[i]) < 1e-2, nm
        for e in range(E):
            want = T.orthogonalize(got[e], [MUON_COEFFS] * 5)
            d = f64(host_bf16(step.dirs[i][e]))
            # the tolerance of the orthogonalisation's own tests
            assert np.linalg.norm(d - want) <= (2.0 ** -8 + 4e4 * 2.0 ** -24) * np.linalg.norm(want)

    # differences of the loss in float64, nothing rounded and the choice held
    def loss(xv, lv):
        p = T.scores(lv, score)
        q = np.take_along_axis(p, ids, -1)
        wv = (1.5 * q / q.sum(-1, keepdims=True)).reshape(R * S, K)
        total = 0.0
        for e in range(E):
            t, k = np.nonzero(it == e)
            if t.size:
                _, yv = swiglu.forward(xv[t], *(f64(h[e]) for h in home_h))
                total += (wv[t, k][:, None] * yv * f64(dt[t])).sum()
        return total

    rng = np.random.default_rng(2)
    x64, l64 = f64(xt), logits.astype(np.float64)
    for which, grad, base in (("logits", got_dl, l64), ("x", f64(host_bf16(step.dx)).reshape(R * S, H), x64)):
        # along the gradient itself and a random direction; six stored tensors lie between, each
        # rounded by at most 2^-8 of itself
        for v in (grad / np.linalg.norm(grad), rng.standard_normal(base.shape)):
            h = 1e-4
            if which == "logits":
                fd = (loss(x64, l64 + h * v) - loss(x64, l64 - h * v)) / (2 * h)
            else:
                fd = (loss(x64 + h * v, l64) - loss(x64 - h * v, l64)) / (2 * h)
            tol = 6 * 2.0 ** -8 * np.linalg.norm(grad) * np.linalg.norm(v)
            assert abs((grad * v).sum() - fd) <= tol, which
    step.buf.destroy()


def test_step_graph_replays_equal_eager():
    w, home_h, x, logits, dout, form = case("sigmoid")
    step = Step(w, [dev_bf16(h) for h in home_h], **form)
    tx, tl, td = dev_bf16(x), dev(logits), dev_bf16(dout)
    perm = torch.randperm(w.S, generator=torch.Generator().manual_seed(1)).cuda()
    ins = [(tx.clone(), tl.clone(), td.clone()), (tx[:, perm], tl.flip(-1), td[:, perm]),
           (tx.flip(0), tl * 2, td.clone())]
    refs = []
    for a in ins:
        step(*[v.contiguous() for v in a])
        torch.cuda.synchronize()
        refs.append([t.clone() for t in step.results()])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(tx, tl, td)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(tx, tl, td)
    for rep in range(2):
        for a, ref in zip(ins, refs):
            for t, v in zip((tx, tl, td), a):
                t.copy_(v)
            for t in step.results():
                t.fill_(1)
            graph.replay()
            torch.cuda.synchronize()
            for i, (t, r) in enumerate(zip(step.results(), ref)):
                assert torch.equal(t, r), i
            tx.add_(0)
            torch.cuda.synchronize()
    del graph
    step.buf.destroy()
