"""moonep_route and moonep_route_bwd at the limits of fp32: chosen sigmoids that
are nearly zero, softmax sums whose additions all round one way, biases that
are not finite."""
import numpy as np
import pytest
import torch

from grouped_gemm_moonep_amd import Buffer
from gpu_util import log
from oracle import training as T

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def tiny_sigmoid_units(K):
    """Roundings, in units of 2^-24, of a normalised weight s_k / t of sigmoids
    below 2^-115: 2 for the exponential, 2 for the sum with 1 and the division, 4
    for a result below 2^-126 (multiples of 2^-149 from 2^-128 on), K more for
    the sum t of them, and 3 for its inverse and the products."""
    return 8 + (8 + K) + 3


@pytest.mark.parametrize("shape", [(1, 33, 2, 8), (2, 9, 8, 64), (3, 5, 20, 129), (2, 11, 8, 384),
                                   (1, 7, 32, 512), (1, 3, 32, 1024)], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1.0, 20.0, 500.0])
def test_gradient_of_sigmoids_near_zero(shape, dtype, size):
    """Every logit so low that the inverse of the chosen sigmoids' sum is 2^115
    .. 2^128: the weights are ordinary and so are the gradients."""
    R, S, K, E = shape
    g = gen(E + K)
    x = (-80 - 8.5 * torch.rand((R, S, E), generator=g, device="cuda")).to(dtype)
    drw = size * torch.randn((R, S, K), generator=g, device="cuda")
    drw[0, 0] = size                                     # equal: no gradient but the rounding's
    buf = Buffer(R=R, S=S, K=K, E=E, H=64, Hp=64)
    form = dict(score="sigmoid", normalize=True, scale=2.5)
    ids, w = buf.route(x, **form)
    d = buf.route_bwd(x, ids, drw, **form)
    buf.destroy()
    log(f"sigmoids near zero {shape} {dtype} drw {size}")
    x64, dw = x.double().cpu().numpy(), drw.double().cpu().numpy()
    want_ids, want_w = T.route(x64, K, **form)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    unit = tiny_sigmoid_units(K)
    err = np.abs(w.double().cpu().numpy() - want_w)
    assert (err <= (unit + 1) * U * want_w).all(), (err / want_w).max() / U
    # (g_k - sum_j g_j w_j) w_k: the weights sum to 1, so the sum is off by a weight's roundings,
    # its products' and its additions', the difference is at most twice the largest g
    want = T.route_bwd(x64, want_ids, dw, **form)
    tol = 2.5 * np.abs(dw).max(-1, keepdims=True) * U * (3 * unit + K + 12)
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    got = d.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()


def test_gradient_of_two_equal_sigmoids_near_zero():
    buf = Buffer(R=1, S=2, K=2, E=8, H=64, Hp=64)
    x = torch.full((1, 2, 8), -88.0, device="cuda")
    x[0, 0] = -87.0
    ids, w = buf.route(x, score="sigmoid")
    assert (w == 0.5).all()
    drw = torch.tensor([[[20.0, -20.0], [4.0, -4.0]]], device="cuda")
    d = buf.route_bwd(x, ids, drw, score="sigmoid")
    buf.destroy()
    want = torch.zeros_like(d)
    want[0, 0, :2] = torch.tensor([10.0, -10.0])
    want[0, 1, :2] = torch.tensor([2.0, -2.0])
    assert torch.allclose(d, want, rtol=16 * U, atol=0)


@pytest.mark.parametrize("dtype,E", [(torch.float32, 256), (torch.float32, 384), (torch.float32, 452),
                                     (torch.float32, 512), (torch.float32, 1024),
                                     (torch.bfloat16, 130), (torch.bfloat16, 384),
                                     (torch.bfloat16, 392), (torch.bfloat16, 512),
                                     (torch.bfloat16, 600)])
@pytest.mark.parametrize("K", [1, 8, 9])
def test_choice_by_a_softmax_whose_sum_rounds_up_throughout(dtype, E, K):
    """One score near one, and 2^-24 of it for every other expert of its lane (16
    bytes of every 256) and for one of each lane that its sum meets: each
    addition to the sum rounds up.  The score with its bias stands a few units of
    2^-24 above that of an expert with hardly a score, whose bias alone decides."""
    R, S = 1, 3
    per = 16 // torch.empty((), dtype=dtype).element_size()
    low = -16.625 if dtype == torch.bfloat16 else float(np.log(1.02 * U))
    buf = Buffer(R=R, S=S, K=K, E=E, H=64, Hp=64)
    lane = (np.arange(E) // per) % 16
    for lead in (0, per - 1, 5 * per, 16 * per):
        x = np.full((R, S, E), -100.0)
        mine = lane == lane[lead]
        for q in (1, 2, 4, 8):
            mine[np.flatnonzero(lane == lane[lead] ^ q)[0]] = True
        x[..., mine] = low
        x[..., lead] = 0
        x = torch.from_numpy(x).to(dtype).cuda()
        other = int(np.flatnonzero(~mine)[-1])
        score = 1 - T.scores(x.double().cpu().numpy(), "softmax")[0, 0, lead]
        for gap in range(-60, 61, 4):                    # units of 2^-24 between the two keys
            bias = torch.full((E,), -10.0, device="cuda")
            bias[lead] = -1
            bias[other] = -score - (gap + 0.5) * U
            want, w = T.route(x.double().cpu().numpy(), K, bias.double().cpu().numpy())
            ids, rw = buf.route(x, bias)
            assert np.array_equal(ids.cpu().numpy(), want), (lead, gap)
            # 64 units for sums, products and exponentials, 2 for each of an argument of up to 100
            assert np.allclose(rw.cpu().numpy(), w, rtol=(64 + 200) * U, atol=1e-30)
    buf.destroy()


@pytest.mark.parametrize("E,K", [(16, 4), (64, 8), (129, 3), (256, 8), (384, 8), (512, 8), (300, 12),
                                 (1024, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("close", [False, True])
def test_a_bias_that_is_not_finite(E, K, score, close):
    """Open experts with a NaN bias first, by their ids, then those with +inf,
    last the closed ones and those with -inf, whether or not the other scores
    are so close that they are compared in 64 bits."""
    S = 9
    g = gen(E)
    x = 0.5 * torch.randn((1, S, E), generator=g, device="cuda")
    bias = 0.3 * torch.randn((E,), generator=g, device="cuda")
    if close:
        x, bias = x.round(), torch.zeros_like(bias)
    odd = torch.randperm(E, generator=g, device="cuda")[:7].tolist()
    bias[odd[:2]] = float("nan")
    bias[odd[2]] = -float("nan")
    bias[odd[3:5]] = float("inf")
    bias[odd[5]] = -float("inf")
    x[0, 1::3, odd[0]] = -float("inf")                   # closed all the same
    x[0, 2, :] = -float("inf")
    x[0, 2, odd[1:4]] = 0.5
    x64 = x.double().cpu().numpy()
    key = T.scores(x64, score) + bias.double().cpu().numpy()
    key = np.where(np.isposinf(key), 1e300, key)
    key = np.where(np.isnan(key), np.inf, key)
    key[np.isneginf(x64)] = -np.inf
    want = np.argsort(-key, axis=-1, kind="stable")[..., :K]
    buf = Buffer(R=1, S=S, K=K, E=E, H=64, Hp=64)
    ids, w = buf.route(x, bias, score=score, normalize=False)
    buf.destroy()
    assert np.array_equal(ids.cpu().numpy(), want)
    want_w = np.take_along_axis(T.scores(x64, score), want, -1)
    assert np.allclose(w.cpu().numpy(), want_w, rtol=80 * U, atol=0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("biased", [False, True])
def test_where_sigmoids_count_as_zero(dtype, biased):
    """The sigmoid in fp32 is 0 from -88.73 down: a token with no other has weights and
    gradients of 0, one with a logit on the other side has them of that one alone."""
    S, E, K = 4, 40, 4
    above, below = (-88.5, -89.0) if dtype == torch.bfloat16 else (-88.72, -88.73)
    x = torch.full((1, S, E), below, device="cuda")
    x[0, 1] = above
    x[0, 2, 7] = above
    x[0, 3, :36] = -float("inf")
    bias = torch.zeros((E,), device="cuda") if biased else None
    buf = Buffer(R=1, S=S, K=K, E=E, H=64, Hp=64)
    ids, w = buf.route(x.to(dtype), bias, score="sigmoid", scale=2.0)
    drw = torch.tensor([9.0, -9.0, 5.0, 1.0], device="cuda").expand(1, S, K).contiguous()
    d = buf.route_bwd(x.to(dtype), ids, drw, score="sigmoid", scale=2.0)
    buf.destroy()
    assert not w[0, [0, 3]].any() and not d[0, [0, 3]].any()
    assert ids[0, 2, 0] == 7 and w[0, 2].tolist() == [2.0, 0.0, 0.0, 0.0] and not d[0, 2].any()
    assert torch.allclose(w[0, 1], torch.full((K,), 0.5, device="cuda"), rtol=16 * U, atol=0)
    want = 2 * (drw[0, 1] - 1.5) / K
    got = d[0, 1, ids[0, 1].long()].float()
    tol = 2.0 ** -8 * want.abs() + (3 * tiny_sigmoid_units(K) + K + 12) * U * 18
    assert (got - want).abs().le(tol).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_equal_in_64_bits_go_by_expert(score):
    """A sigmoid of 41 is above one of 40, and a softmax of -800 above one of -900,
    but not in 64 bits."""
    x = torch.full((1, 1, 32), -50.0 if score == "sigmoid" else -1000.0, device="cuda")
    high = (40.0, 41.0, 42.0) if score == "sigmoid" else (-900.0, -850.0, -800.0)
    x[0, 0, [5, 11, 30]] = torch.tensor(high, device="cuda")
    x[0, 0, 20] = 39.9 if score == "sigmoid" else 0.0
    buf = Buffer(R=1, S=1, K=4, E=32, H=64, Hp=64)
    bias = torch.zeros((32,), device="cuda")
    bias[[5, 11, 30]] = 0.25
    ids, _ = buf.route(x, bias, score=score)
    buf.destroy()
    want = [5, 11, 30, 20] if score == "sigmoid" else [20, 5, 11, 30]
    assert ids[0, 0].tolist() == want


@pytest.mark.parametrize("E,K", [(16, 4), (64, 8), (256, 8), (384, 8), (300, 12), (1024, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_softmax_without_scores_goes_by_its_logits(E, K, dtype):
    """Rows with a NaN or +inf beside ordinary ones: NaN logits and biases first, then +inf,
    then the other logits, whatever their biases."""
    S = 8
    g = gen(E)
    x = torch.randn((1, S, E), generator=g, device="cuda").to(dtype)
    bias = torch.randn((E,), generator=g, device="cuda")
    odd = torch.randperm(E, generator=g, device="cuda")[:6].tolist()
    bias[odd[0]] = float("nan")
    bias[odd[1]] = -float("inf")
    x[0, 1::2, odd[2]] = float("inf")
    x[0, 2::4, odd[3]] = float("nan")
    x[0, 1::2, odd[4]] = -float("inf")
    x64 = x.double().cpu().numpy()
    b64 = bias.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        key = T.scores(x64, "softmax") + b64
    rows = ~np.isfinite(np.where(np.isneginf(x64), 0, x64)).all(-1)
    key[rows] = x64[rows]
    key = np.where(np.isposinf(key), 1e300, key)
    key = np.where(np.isnan(key) | np.isnan(b64), np.inf, key)
    key[np.isneginf(x64)] = -np.inf
    want = np.argsort(-key, axis=-1, kind="stable")[..., :K]
    buf = Buffer(R=1, S=S, K=K, E=E, H=64, Hp=64)
    ids, _ = buf.route(x, bias)
    buf.destroy()
    assert rows.sum() == 6 and np.array_equal(ids.cpu().numpy(), want)
