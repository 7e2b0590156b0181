"""moonep_route and moonep_route_bwd on the GPU against the oracle's router in
64 bits: ids equal, weights and gradients within a bound counted in roundings;
ties, closed experts, NaN, close scores, in-place gradients, graph replays and
refusals."""
import numpy as np
import pytest
import torch

from grouped_gemm_moonep_amd import Buffer, MoonepError
from gpu_util import log
from oracle import training as T

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def make(R, S, K, E):
    return Buffer(R=R, S=S, K=K, E=E, H=64, Hp=64)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def weight_tolerance(x, ids, w):
    """Units of rounding in a weight: at most 32 additions per lane and 6
    between lanes in a sum, under 16 for exponentials, quotients and products, and
    the rounding of the exponent's argument, which grows with its size."""
    far = np.abs(np.take_along_axis(x, ids, -1)) + np.abs(np.where(np.isfinite(x), x, 0)).max(-1, keepdims=True)
    return (64 + 2 * np.where(np.isfinite(far), far, 0)) * U * np.abs(w)


def check(logits, bias, K, score, normalize, scale, drw=None):
    R, S, E = logits.shape
    buf = make(R, S, K, E)
    form = dict(score=score, normalize=normalize, scale=scale)
    ids, w = buf.route(logits, bias, **form)
    x = logits.double().cpu().numpy()
    want_ids, want_w = T.route(x, K, None if bias is None else bias.double().cpu().numpy(), **form)
    got_ids = ids.cpu().numpy()
    assert np.array_equal(got_ids, want_ids), f"{(got_ids != want_ids).sum()} ids differ"
    err = np.abs(w.cpu().numpy() - want_w)
    assert np.all(err <= weight_tolerance(x, want_ids, want_w)), err.max()
    if drw is None:
        drw = torch.randn((R, S, K), generator=gen(7), device="cuda")
    d = buf.route_bwd(logits, ids, drw, **form)
    assert d.dtype == logits.dtype
    gw = drw.double().cpu().numpy()
    want = T.route_bwd(x, want_ids, gw, **form)
    # what the sums in a row are made of, times their roundings; then the output's own
    size = scale * np.abs(gw).max(-1, keepdims=True) * (want_ids.shape[-1] + 2)
    far = np.where(np.isfinite(x), np.abs(x), 0).max(-1, keepdims=True)
    tol = (128 + 4 * far) * U * size
    if logits.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    err = np.abs(d.float().cpu().numpy() - want)
    assert np.all(err <= tol), (err / tol).max()
    buf.destroy()


SHAPES = [(1, 1, 1, 1), (1, 1, 1, 8), (2, 3, 2, 6), (1, 5, 8, 8), (4, 16, 4, 32), (1, 33, 32, 33),
          (8, 9, 8, 64), (1, 17, 20, 65), (2, 31, 7, 130), (1, 12, 32, 128), (8, 37, 8, 256),
          (3, 11, 9, 255), (1, 7, 32, 256), (8, 13, 8, 384), (2, 5, 10, 384), (1, 9, 8, 500),
          (4, 3, 6, 512), (1, 5, 32, 512), (1, 6, 8, 513), (2, 4, 32, 1024)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False),
                                             ("sigmoid", True), ("sigmoid", False)])
def test_route_matches_oracle(shape, score, normalize):
    R, S, K, E = shape
    log(f"route {shape} {score} normalize={normalize}")
    g = gen(E * 37 + K)
    for dtype in (torch.float32, torch.bfloat16):
        x = (2 * torch.randn((R, S, E), generator=g, device="cuda")).to(dtype)
        b = 0.1 * torch.randn((E,), generator=g, device="cuda")
        for bias in (None, b):
            check(x, bias, K, score, normalize, 2.5)


@pytest.mark.parametrize("E,K", [(64, 6), (256, 8), (384, 8), (300, 12)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["equal", "few_values", "zero_bias", "saturated", "shared_score"])
def test_ties_and_close_scores(E, K, score, kind):
    """Equal scores go to the lower expert, and scores closer than their
    rounding in 32 bits to the exactly larger one: more of them than a row has
    lanes, too."""
    log(f"ties E={E} K={K} {score} {kind}")
    g = gen(E + K)
    x = torch.randn((2, 25, E), generator=g, device="cuda")
    bias = 0.1 * torch.randn((E,), generator=g, device="cuda")
    if kind == "equal":
        x.zero_()
        bias = None
    elif kind == "few_values":
        x = x.round()
        bias = None
    elif kind == "zero_bias":
        x = x.bfloat16()
        bias.zero_()
    elif kind == "saturated":
        x = 12 + 6 * x                      # sigmoids within 1e-5 of one, many closer than 2^-24
        bias.zero_()
    else:
        x = x * 1e-6                        # every score within 1e-6 of every other
        bias = torch.zeros_like(bias)
    check(x, bias, K, score, True, 1.0)


@pytest.mark.parametrize("K", [5, 8])
@pytest.mark.parametrize("E", [256, 384, 512])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ahead", [0, 4, 7, 8])
def test_best_experts_of_one_lane_are_close(E, K, dtype, ahead):
    """Experts that one lane reads (16 bytes of every 256), of which `ahead` lead and the others
    have one score in 32 bits and exact ones that rise with the expert: more candidates
    than the lane keeps, and the last of them is the right one."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    mine = [e for e in range(E) if e // per % 16 == 3]
    x = torch.full((1, 3, E), -6.0, device="cuda")
    x[..., mine] = 1.0
    x[..., mine[:ahead]] = 3.0
    bias = torch.zeros((E,), device="cuda")
    bias[mine] = torch.arange(1, len(mine) + 1, device="cuda") * 2.0 ** -30
    check(x.to(dtype), bias, K, "sigmoid", True, 1.0)
    check(x.to(dtype), bias, K, "softmax", True, 1.0)


@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False),
                                             ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("biased", [False, True])
def test_closed_experts(score, normalize, biased):
    g = gen(11)
    x = torch.randn((2, 40, 96), generator=g, device="cuda")
    x[torch.rand(x.shape, generator=g, device="cuda") < 0.9] = -float("inf")
    x[0, 0] = -float("inf")                          # no open expert
    x[0, 1, :95] = -float("inf")                     # one
    bias = torch.rand((96,), generator=g, device="cuda") if biased else None
    check(x, bias, 8, score, normalize, 1.5)


def test_infinite_and_nan_logits_show_and_stay_in_their_row():
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn((1, 6, 48), generator=gen(3), device="cuda").to(dtype)
        clean = x.clone()
        x[0, 1, 17] = float("nan")
        x[0, 3, 20] = -float("nan")
        x[0, 4, 5] = float("inf")
        x[0, 4, 40] = float("nan")
        buf = make(1, 6, 4, 48)
        for bias in (None, torch.zeros(48, device="cuda")):
            for score in ("softmax", "sigmoid"):
                ids, w = buf.route(x, bias, score=score)
                ref, wr = buf.route(clean, bias, score=score)
                assert ids[0, 1, 0] == 17 and ids[0, 3, 0] == 20
                assert torch.isnan(w[0, [1, 3, 4], 0]).all()
                assert ids[0, 4, :2].tolist() == [40, 5]
                for s in range(6):
                    assert len(set(ids[0, s].tolist())) == 4 and 0 <= ids[0, s].min()
                keep = [0, 2, 5]
                assert torch.equal(ids[0, keep], ref[0, keep])
                assert torch.equal(w[0, keep], wr[0, keep])
        buf.destroy()


def test_unaligned_rows_given_outputs_and_in_place_gradient():
    """Rows that do not start on 16 bytes, outputs of the caller, dlogits in
    logits' storage, another stream."""
    R, S, K, E = 2, 19, 5, 36
    store = torch.randn(R * S * E + 1, generator=gen(4), device="cuda")
    x = store[1:].view(R, S, E)
    y = x.clone()
    buf = make(R, S, K, E)
    ids, w = buf.route(y)
    topk, rw = torch.empty_like(ids), torch.empty_like(w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = buf.route(x, topk=topk, rw=rw)
        assert got[0] is topk and got[1] is rw
        drw = torch.ones_like(rw)
        drw[..., 0] = 3
        want = buf.route_bwd(y, topk, drw, normalize=False)
        out = buf.route_bwd(x, topk, drw, normalize=False, dlogits=x)
    torch.cuda.current_stream().wait_stream(side)
    assert out is x and torch.equal(ids, topk) and torch.equal(w, rw)
    assert torch.equal(x, want)
    buf.destroy()


def test_backward_leaves_out_foreign_ids():
    buf = make(1, 2, 2, 16)
    x = torch.randn((1, 2, 16), generator=gen(5), device="cuda")
    drw = torch.ones((1, 2, 2), device="cuda")
    ids = torch.tensor([[[3, 16], [-1, 2 ** 30]]], dtype=torch.int32, device="cuda")
    d = buf.route_bwd(x, ids, drw, score="sigmoid", normalize=False)
    assert torch.count_nonzero(d) == 1 and d[0, 0, 3] > 0
    buf.destroy()


def test_graph_replays_equal_eager():
    buf = make(4, 65, 8, 256)
    x = torch.empty((4, 65, 256), device="cuda")
    bias = 0.05 * torch.randn((256,), generator=gen(1), device="cuda")
    drw = torch.randn((4, 65, 8), generator=gen(2), device="cuda")
    topk = torch.empty((4, 65, 8), dtype=torch.int32, device="cuda")
    rw = torch.empty((4, 65, 8), device="cuda")
    d = torch.empty_like(x)

    def step():
        buf.route(x, bias, score="sigmoid", topk=topk, rw=rw)
        buf.route_bwd(x, topk, drw, score="sigmoid", dlogits=d)

    ins = [torch.randn(x.shape, generator=gen(s), device="cuda") for s in range(3)]
    refs = []
    for v in ins:
        x.copy_(v)
        step()
        refs.append([t.clone() for t in (topk, rw, d)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(2):
        for v, ref in zip(ins, refs):
            x.copy_(v)
            for t in (topk, rw, d):
                t.fill_(1)
            graph.replay()
            torch.cuda.synchronize()
            for t, r in zip((topk, rw, d), ref):
                assert torch.equal(t, r)
            x.add_(1)
            torch.cuda.synchronize()
    del graph
    buf.destroy()


def test_refusals():
    buf = make(2, 4, 2, 8)
    x = torch.zeros((2, 4, 8), device="cuda")
    ids = torch.zeros((2, 4, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((2, 4, 2), device="cuda")
    for bad, kind in [(dict(logits=x.half()), TypeError), (dict(logits=x[:1]), ValueError),
                      (dict(logits=x.cpu()), ValueError),
                      (dict(logits=x.new_zeros((4, 2, 8)).transpose(0, 1)), ValueError),
                      (dict(logits=x, bias=torch.zeros(7, device="cuda")), ValueError),
                      (dict(logits=x, bias=torch.zeros(8).double().cuda()), TypeError),
                      (dict(logits=x, score="relu"), ValueError),
                      (dict(logits=x, rw=x.view(-1)[:16].view(2, 4, 2)), ValueError),
                      (dict(logits=x, topk=w.view(torch.int32), rw=w), ValueError),
                      (dict(logits=x, topk=ids.long()), TypeError)]:
        with pytest.raises(kind):
            buf.route(**bad)
    for bad, kind in [(dict(topk=ids.long(), drw=w), TypeError), (dict(topk=ids, drw=None), ValueError),
                      (dict(topk=ids, drw=w, dlogits=x.bfloat16()), TypeError),
                      (dict(topk=ids, drw=w, dlogits=x[..., :4]), ValueError)]:
        with pytest.raises(kind):
            buf.route_bwd(x, **bad)
    from grouped_gemm_moonep_amd import _abi, lib
    p = x.data_ptr()
    assert lib().moonep_route(buf._h, p, 7, None, 0, 1, 1.0, ids.data_ptr(), w.data_ptr(),
                              None) == _abi.MOONEP_ERR_ARG
    assert lib().moonep_route(buf._h, p + 2, 0, None, 0, 1, 1.0, ids.data_ptr(), w.data_ptr(),
                              None) == _abi.MOONEP_ERR_ARG
    assert lib().moonep_route(buf._h, p, 0, None, 2, 1, 1.0, ids.data_ptr(), w.data_ptr(),
                              None) == _abi.MOONEP_ERR_ARG
    assert lib().moonep_route_bwd(buf._h, p, 0, 0, 1, 1.0, ids.data_ptr(), w.data_ptr(), None,
                                  None) == _abi.MOONEP_ERR_ARG
    buf.destroy()
    with pytest.raises(MoonepError):                  # a destroyed handle
        buf.route(x)
