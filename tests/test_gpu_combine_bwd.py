"""moonep_combine_bwd on the GPU against the oracle: slot gradients bit-exact
(bf16 of the fp32 product), route-weight gradients within the roundings of
their sum; every row width class, in place, without drw, CU budgets, slots
behind the last segment untouched, no-op plans, graph replays, refusals."""
import ctypes

import numpy as np
import pytest
import torch

import moonep_synth as synth
import oracle
from gpu_util import buffer_for, dev, dev_bf16, host_bf16, log
from grouped_gemm_moonep_amd import _abi, lib
from oracle import training as T

pytestmark = pytest.mark.gpu

FILL = 0x7E55


def inputs(w, target, W, seed=3):
    topk, _ = synth.routing(w, target)
    p = oracle.plan(topk, w.E, w.B, w.token_padding)
    rng = np.random.default_rng(seed)
    y = synth.to_bf16_bits(rng.standard_normal((w.R, p.NvS, W), dtype=np.float32))
    d = synth.to_bf16_bits(rng.standard_normal((w.R, w.S, W), dtype=np.float32))
    rw = rng.standard_normal((w.R, p.NvS), dtype=np.float32)
    return topk, p, y, d, rw


def filled(shape):
    return torch.full(shape, FILL, dtype=torch.int16, device="cuda").view(torch.bfloat16)


def sum_bound(W, bound):
    """Additions in a lane (8 per vector it holds) and between lanes, each off
    by 2^-24 of at most the sum of the products' magnitudes."""
    lanes = next(g for g in (8, 16, 32, 64) if g >= W // 8 or g == 64)
    return (8 * -(-(W // 8) // lanes) + 6) * 2.0 ** -24 * bound


def check(w, target, W, num_cus=0, in_place=False, need_drw=True):
    log(f"combine_bwd {w.name} target={target} W={W} cus={num_cus} in_place={in_place}")
    topk, p, y, d, rw = inputs(w, target, W)
    buf = buffer_for(w, num_cus=num_cus)
    plan = buf.plan(dev(topk))
    ty = dev_bf16(y)
    out = ty if in_place else filled(y.shape)
    dy, drw = buf.combine_bwd(plan, dev_bf16(d), ty if need_drw else None, dev(rw), dy_nvs=out,
                              need_drw=need_drw)
    assert dy is out
    want_dy, want, bound = T.combine_bwd(p, d, y, rw)
    got = host_bf16(dy)
    for r in range(w.R):
        end = p.cu_seqlens[r, -1]
        assert np.array_equal(got[r, :end], want_dy[r, :end])
        assert np.array_equal(got[r, end:], y[r, end:] if in_place else np.full_like(got[r, end:], FILL))
    if need_drw:
        err = np.abs(drw.cpu().numpy() - want)
        assert np.all(err <= sum_bound(W, bound)), (err / sum_bound(W, bound)).max()
    else:
        assert drw is None
    buf.destroy()


@pytest.mark.parametrize("name,target", [
    (n, t) for n, ts in synth.SWEEPS.items() for t in ts if n.startswith(("tiny", "mid"))]
    + [("tiny_r4_s64_k2_e8", "adv"), ("mid_r8_s1024_k4_e32", "adv")])
def test_matches_oracle(name, target):
    w = synth.WORKLOADS[name]
    check(w, target, w.H)


@pytest.mark.parametrize("width", [8, 16, 64, 72, 128, 136, 248, 264, 512, 520, 1032, 4104])
@pytest.mark.parametrize("in_place", [False, True])
def test_row_widths(width, in_place):
    check(synth.WORKLOADS["tiny_r4_s64_k2_e8"], 1.0, width, in_place=in_place)


@pytest.mark.parametrize("kw", [dict(num_cus=1), dict(num_cus=3), dict(need_drw=False),
                                dict(num_cus=2, in_place=True)])
@pytest.mark.parametrize("width", [40, 1024])
def test_cu_budget_and_no_weight_gradient(kw, width):
    check(synth.WORKLOADS["tiny_r4_s64_k2_e8"], 1.0, width, **kw)


def test_inference_prefetch_rows():
    """B < E/R: remote experts beyond B sit in their home rows."""
    w = synth.WORKLOADS["infer_r8_s128_k8_e256_b4"]
    check(w, 4.0, 200)


def test_headline_sampled():
    w = synth.WORKLOADS["fwd_r8_s4096_k8_e256"]
    topk, _ = synth.routing(w, 1.0)
    log("combine_bwd headline sampled")
    p = oracle.plan(topk, w.E, w.B, w.token_padding)
    g = torch.Generator(device="cuda").manual_seed(5)
    y = torch.randn((w.R, p.NvS, w.H), generator=g, device="cuda").to(torch.bfloat16)
    d = torch.randn((w.R, w.S, w.H), generator=g, device="cuda").to(torch.bfloat16)
    rw = torch.rand((w.R, p.NvS), generator=g, device="cuda")
    buf = buffer_for(w)
    plan = buf.plan(dev(topk))
    out = filled(y.shape)
    dy, drw = buf.combine_bwd(plan, d, y, rw, dy_nvs=out)
    dest = dev(p.dest.reshape(-1))
    want = (rw.view(-1)[dest].view(-1, w.K, 1) * d.view(-1, 1, w.H).float()).bfloat16()
    assert torch.equal(dy.view(-1, w.H)[dest].view(-1, w.K, w.H).view(torch.int16),
                       want.view(torch.int16))
    del want
    toks = torch.arange(0, w.R * w.S, 97, device="cuda")
    a = d.view(-1, w.H)[toks].double()
    b = y.view(-1, w.H)[dest.view(-1, w.K)[toks]].double()
    prod = a[:, None] * b
    err = (drw.view(-1, w.K)[toks].double() - prod.sum(-1)).abs()
    assert (err <= torch.from_numpy(sum_bound(w.H, prod.abs().sum(-1).cpu().numpy())).cuda()).all()
    used = torch.zeros(w.R * p.NvS, dtype=torch.bool, device="cuda")
    used[dest] = True
    for r in range(w.R):
        end = int(p.cu_seqlens[r, -1])
        rows = dy[r].view(torch.int16)
        pad = ~used[r * p.NvS:r * p.NvS + end]
        assert not rows[:end][pad].any()
        assert (rows[end:] == FILL).all()
    buf.destroy()


def test_no_op_plan_of_a_bad_routing_stays_in_bounds():
    w = synth.WORKLOADS["tiny_r4_s64_k2_e8"]
    topk = synth.routing(w, 1.0)[0].copy()
    topk[1, 5, 0] = w.E + 3
    buf = buffer_for(w)
    plan = buf.plan(dev(topk))
    assert buf.read_stats(plan)[0] != 0
    y = torch.ones((w.R, buf.NvS, 64), dtype=torch.bfloat16, device="cuda")
    d = torch.ones((w.R, w.S, 64), dtype=torch.bfloat16, device="cuda")
    dy, drw = buf.combine_bwd(plan, d, y, torch.ones((w.R, buf.NvS), device="cuda"))
    assert torch.isfinite(drw).all() and dy.shape == y.shape
    buf.destroy()


def test_results_do_not_depend_on_the_launch_and_graph_replays_equal_eager():
    w = synth.WORKLOADS["tiny_r4_s64_k2_e8"]
    topk, p, y, d, rw = inputs(w, 1.0, 264)
    a, b = buffer_for(w), buffer_for(w, num_cus=1)
    ins = [dev_bf16(d), dev_bf16(y), dev(rw)]
    pa, pb = a.plan(dev(topk)), b.plan(dev(topk))
    da, wa = a.combine_bwd(pa, *ins, dy_nvs=filled(y.shape))
    db, wb = b.combine_bwd(pb, *ins, dy_nvs=filled(y.shape))
    assert torch.equal(da.view(torch.int16), db.view(torch.int16)) and torch.equal(wa, wb)
    out, drw = filled(y.shape), torch.empty_like(wa)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.combine_bwd(pa, *ins, dy_nvs=out, drw=drw)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.combine_bwd(pa, *ins, dy_nvs=out, drw=drw)
    for f in (1.0, 2.0, -0.5):
        ins[0].copy_(dev_bf16(d).float() * f)                # a power of two: exact
        out.view(torch.int16).fill_(FILL)
        drw.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        ref = a.combine_bwd(pa, *ins, dy_nvs=filled(y.shape))
        assert torch.equal(out.view(torch.int16), ref[0].view(torch.int16))
        assert torch.equal(drw, ref[1]) and torch.equal(drw, wa * f)
        torch.cuda.synchronize()
    del graph
    a.destroy()
    b.destroy()


def test_refusals():
    w = synth.WORKLOADS["tiny_r4_s64_k2_e8"]
    topk, p, y, d, rw = inputs(w, 1.0, 64)
    buf = buffer_for(w)
    plan = buf.plan(dev(topk))
    y, d, rw = dev_bf16(y), dev_bf16(d), dev(rw)
    for bad, kind in [(dict(dout=d.float()), TypeError), (dict(dout=d[:, :-1]), ValueError),
                      (dict(y_nvs=None), ValueError), (dict(y_nvs=y[..., :32]), ValueError),
                      (dict(rw_nvs=None), ValueError), (dict(rw_nvs=rw.double()), TypeError),
                      (dict(rw_nvs=rw.cpu()), ValueError),
                      (dict(need_drw=False, drw=torch.zeros((w.R, w.S, w.K), device="cuda")), ValueError),
                      (dict(drw=torch.zeros((w.R, w.S, w.K + 1), device="cuda")), ValueError),
                      (dict(drw=rw.view(-1)[:w.R * w.S * w.K].view(w.R, w.S, w.K)), ValueError)]:
        args = dict(dout=d, y_nvs=y, rw_nvs=rw)
        args.update(bad)
        with pytest.raises(kind):
            buf.combine_bwd(plan, **args)
    big = torch.zeros(y.numel() + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="overlap"):           # shifted over its input
        buf.combine_bwd(plan, d, big[8:].view(y.shape), rw, dy_nvs=big[:-8].view(y.shape))
    call = lambda W, dout, yy, r, dy, dr: lib().moonep_combine_bwd(
        buf._h, ctypes.byref(plan.struct), dout, W, yy, r, dy, dr, None)
    ok = [64, d.data_ptr(), y.data_ptr(), rw.data_ptr(), big.data_ptr(), rw.data_ptr()]
    for i, v in [(0, 0), (0, 12), (1, None), (1, ok[1] + 2), (2, None), (2, ok[2] + 8), (3, None),
                 (3, ok[3] + 1), (4, None), (4, ok[4] + 2), (4, ok[1]), (5, ok[5] + 2)]:
        a = list(ok)
        a[i] = v
        assert call(*a) == _abi.MOONEP_ERR_ARG, (i, v)
    buf.destroy()
