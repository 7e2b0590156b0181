"""block_norm and block_norm_bwd on the GPU against the oracle in float64:
every gate, stream type and combination of norms, rows of one vector to the
widest, one row to many, in place, NaN and infinities, graphs, streams.

Tolerances count roundings: with e = 2^-24 a sum of a row passes at most 16
additions in a lane and 10 between lanes, so a mean of squares is off by at
most 28 e of itself, its rstd by half of that and three roundings more, and a
product with it by under 20 e; each further product or sum adds one e.  A
result in bf16 is off by half a step more (2^-8 of its value)."""
import numpy as np
import pytest
import torch

from gpu_util import log
from grouped_gemm_moonep_amd import (block_norm, block_norm_bwd, block_norm_bwd_workspace)
from oracle import block as B

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
HALF = {torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2, torch.float32: E}
TINY = 1e-30
GATES = [None, "channel", "token", "full"]


def draw(T, W, dtype, gate="channel", two=True, post=True, pre=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    v = dict(y=(n(T, W) * torch.exp(n(T, 1))).bfloat16(), y2=n(T, W).bfloat16() if two else None,
             gate={None: lambda: None, "channel": lambda: n(W), "token": lambda: n(T, 1),
                   "full": lambda: n(T, W).bfloat16()}[gate](),
             w_post=1 + 0.3 * n(W) if post else None, w_pre=1 + 0.3 * n(W) if pre else None)
    return n(T, W).to(dtype), v, n


def wide(t):
    return None if t is None else t.double().cpu().numpy()


def within(got, want, err, what):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, what
    bad = np.abs(got - want) - err
    log(f"{what}: worst error / bound {float((np.abs(got - want) / (err + TINY)).max()) if got.size else 0:.3f}")
    assert not got.size or bad.max() <= 0, f"{what}: {bad.max():.3e} over its bound"


def forward_bounds(h, v, scale, eps):
    """(h', u) and how far each may be off, u before its rounding."""
    o = {k: wide(t) for k, t in v.items()}
    hd = wide(h)
    out, u = B.block_norm(hd, scale=scale, eps=eps, **o)
    term = np.abs(out - hd)
    if o["y"] is not None and o["y2"] is not None and o["w_post"] is None:
        # y + y2 is rounded once, against its parts
        g = 1.0 if o["gate"] is None else np.abs(o["gate"])
        term = scale * g * (np.abs(o["y"]) + np.abs(o["y2"]))
    e_out = E * (24 * term + np.abs(out)) if o["y"] is not None else 0 * out
    if u is None:
        return out, None, e_out, None
    s = B.rstd(out, eps)
    # the row's error reaches its rstd through the mean of squares
    rel = 20 * E + s * s * (np.abs(out) * e_out).mean(-1, keepdims=True)
    return out, u, e_out, np.abs(o["w_pre"]) * s * e_out + np.abs(u) * (rel + 2 * E)


def check_forward(T, W, dtype, scale=0.5, eps=1e-6, **form):
    what = f"block_norm T={T} W={W} {dtype} {form}"
    log(what)
    h, v, _ = draw(T, W, dtype, **form)
    got, u = block_norm(h, scale=scale, eps=eps, **v)
    out, want, e_out, e_u = forward_bounds(h, v, scale, eps)
    assert got.dtype == dtype and (u is None) == (v["w_pre"] is None)
    within(got, out, e_out + HALF[dtype] * (np.abs(out) + e_out), what + " h")
    if u is not None:
        within(u, want, e_u + HALF[torch.bfloat16] * (np.abs(want) + e_u), what + " u")
    return h, v, got, u


def check_backward(T, W, dtype, scale=0.5, eps=1e-6, with_dh=True, **form):
    what = f"block_norm_bwd T={T} W={W} {dtype} {form}"
    log(what)
    h, v, n = draw(T, W, dtype, **form)
    dh = n(T, W).to(dtype) if with_dh else None
    du = n(T, W).bfloat16() if v["w_pre"] is not None else None
    got = block_norm_bwd(h, dh, du, scale=scale, eps=eps, **v)
    o = {k: wide(t) for k, t in v.items()}
    hd, dhd, dud = wide(h), wide(dh), wide(du)
    want = B.block_norm_bwd(hd, dhd, dud, scale=scale, eps=eps, **o)
    shares = block_norm_bwd_workspace(T, W).numel() // (12 * W)
    depth = -(-T // max(shares, 1)) + -(-shares // 16) + 20
    # what each value is summed from, in magnitude
    mag = np.zeros_like(hd) if dhd is None else np.abs(dhd)
    if dud is not None:
        s = B.rstd(hd, eps)
        w = np.abs(dud * o["w_pre"])
        mag = mag + s * (w + np.abs(hd) * s * s * (w * np.abs(hd)).mean(-1, keepdims=True))
    e_d = 60 * E * mag
    within(got[0], want[0], e_d + HALF[dtype] * (np.abs(want[0]) + e_d), what + " dres")
    if dud is not None:
        t = np.abs(dud * hd * s)
        within(got[4], want[4], E * (depth + 24) * t.sum(0), what + " dw_pre")
    if v["y"] is None:
        assert got[1] is None and got[2] is None and got[3] is None
        return got
    a = np.abs(o["y"] if o["y2"] is None else o["y"] + o["y2"])
    a_in = np.abs(o["y"]) + (0 if o["y2"] is None else np.abs(o["y2"]))
    e_a = E * a_in                                    # the rounding of y + y2
    r = 1.0 if o["w_post"] is None else B.rstd(a, eps)
    wp = 1.0 if o["w_post"] is None else np.abs(o["w_post"])
    g = 1.0 if o["gate"] is None else np.abs(o["gate"])
    e_n = r * wp * (e_a + 24 * E * a)
    md = scale * mag                                  # bounds |scale D|
    e_t = md * e_n + scale * e_d * r * wp * a + 4 * E * md * r * wp * a
    if o["gate"] is not None:
        kind = o["gate"].shape
        if kind == hd.shape:
            lim = e_t + HALF[torch.bfloat16] * (np.abs(want[2]) + e_t)
        elif len(kind) == 1:
            lim = (e_t + E * depth * md * r * wp * a).sum(0)
        else:
            lim = (e_t + 30 * E * md * r * wp * a).sum(-1, keepdims=True)
        within(got[2], want[2], lim, what + " dgate")
    e_dn = g * (scale * e_d + 3 * E * md)
    if o["w_post"] is None:
        e_y = e_dn
    else:
        vm, e_v = wp * g * md, wp * e_dn + E * wp * g * md
        m_abs = (vm * a).mean(-1, keepdims=True)
        e_m = (e_v * a + vm * e_a + 30 * E * vm * a).mean(-1, keepdims=True)
        e_y = r * (e_v + a * r * r * (e_m + 60 * E * m_abs) + e_a * r * r * m_abs +
                   30 * E * (vm + a * r * r * m_abs))
        t = g * md * a * r
        within(got[3], want[3], (e_dn * a * r + g * md * r * (e_a + 24 * E * a) +
                                 E * depth * t).sum(0), what + " dw_post")
    within(got[1], want[1], e_y + HALF[torch.bfloat16] * (np.abs(want[1]) + e_y), what + " dy")
    return got


DTYPES = [torch.bfloat16, torch.float32]
# one vector; a wave's one and two vectors a lane, whole and ragged; workgroups of two waves to
# sixteen, whole and ragged; two vectors a lane there, whole and ragged
WIDTHS = [8, 64, 512, 520, 1024, 1032, 2048, 7168, 7176, 8192, 8200, 16384]


@pytest.mark.parametrize("W", WIDTHS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_forward_widths(W, dtype):
    check_forward(5, W, dtype)


@pytest.mark.parametrize("W", WIDTHS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_backward_widths(W, dtype):
    check_backward(5, W, dtype)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 7, 255, 2049, 5000])
@pytest.mark.parametrize("W", [128, 1032])
def test_token_counts(T, W):
    check_forward(T, W, torch.bfloat16, gate="token")
    check_backward(T, W, torch.float32, gate="token")


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("post,pre,two", [(True, True, True), (True, False, False),
                                          (False, True, True), (False, False, True),
                                          (False, True, False)])
@pytest.mark.parametrize("W", [72, 1096])
def test_forms(gate, post, pre, two, W):
    form = dict(gate=gate, post=post, pre=pre, two=two)
    check_forward(37, W, torch.float32, **form)
    check_backward(37, W, torch.bfloat16, **form)


@pytest.mark.parametrize("gate,post,pre", [("channel", True, True), ("channel", False, True),
                                           ("token", True, False), ("full", True, True),
                                           (None, False, False)])
@pytest.mark.parametrize("W,dtype", [(8264, torch.float32), (12288, torch.bfloat16)])
def test_backward_of_wide_rows(gate, post, pre, W, dtype):
    """More rows than CUs: some workgroups sum two rows."""
    check_backward(300, W, dtype, gate=gate, post=post, pre=pre)


def test_no_gradient_from_behind():
    check_backward(9, 264, torch.float32, with_dh=False)


def test_norm_alone():
    h, v, n = draw(11, 2056, torch.bfloat16)
    w = v["w_pre"]
    out, u = block_norm(h, w_pre=w)
    assert out is h
    _, want, _, e = forward_bounds(h, dict(y=None, y2=None, gate=None, w_post=None, w_pre=w), 1.0,
                                   1e-6)
    within(u, want, e + HALF[torch.bfloat16] * (np.abs(want) + e), "norm alone")
    du = n(11, 2056).bfloat16()
    got = block_norm_bwd(h, None, du, w_pre=w)
    ref = B.block_norm_bwd(wide(h), None, wide(du), w_pre=wide(w))
    assert np.linalg.norm(wide(got[0]) - ref[0]) <= 2 ** -8 * np.linalg.norm(ref[0])
    assert np.linalg.norm(wide(got[4]) - ref[4]) <= 1e-5 * np.linalg.norm(ref[4])
    assert got[1:4] == (None, None, None)


@pytest.mark.parametrize("W", [136, 1544])
def test_in_place(W):
    h, v, n = draw(21, W, torch.float32, gate="full")
    want_h, want_u = block_norm(h, **v)
    hh, y2 = h.clone(), v["y2"].clone()
    got_h, got_u = block_norm(hh, v["y"], y2, v["gate"], v["w_post"], v["w_pre"], h_out=hh, u=y2)
    assert got_h is hh and got_u is y2
    assert torch.equal(got_h, want_h) and torch.equal(got_u, want_u)
    dh, du = n(21, W), n(21, W).bfloat16()
    want = block_norm_bwd(h, dh, du, **v)
    d2 = dh.clone()
    for name in ("y", "y2", "du"):
        vv = dict(v, du=du)
        vv[name] = vv[name].clone()
        got = block_norm_bwd(h, d2.copy_(dh), dres=d2, dy=vv[name], **vv)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_tokens_and_no_gradients_of_weights():
    h, v, n = draw(0, 128, torch.float32)
    out, u = block_norm(h, **v)
    assert out.shape == u.shape == (0, 128)
    got = block_norm_bwd(h, h.clone(), u.clone(), **v)
    assert got[0].shape == got[1].shape == (0, 128)
    assert all(not t.any() for t in got[2:])          # sums over no tokens are zeros
    h, v, n = draw(6, 128, torch.float32)
    dh, du = n(6, 128), n(6, 128).bfloat16()
    full, part = block_norm_bwd(h, dh, du, **v), block_norm_bwd(h, dh, du, need_dw=False, **v)
    assert torch.equal(full[0], part[0]) and torch.equal(full[1], part[1])
    assert part[2:] == (None, None, None)


def test_zero_rows_are_finite():
    h, v, n = draw(8, 1032, torch.float32, two=False)
    h[3] = 0
    v["y"][3] = 0
    out, u = block_norm(h, **v)
    assert not out[3].any() and not u[3].any()
    du = n(8, 1032).bfloat16()
    got = block_norm_bwd(h, None, du, **v)
    assert all(torch.isfinite(t).all() for t in got)
    # rstd of a zero row is 1 / sqrt(eps)
    want = du[3].double() * v["w_pre"].double() * 1e3
    assert torch.allclose(got[0][3].double(), want, rtol=1e-6)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("W", [200, 1800])
def test_bad_values_stay_in_their_row(bad, W):
    h, v, n = draw(10, W, torch.float32)
    clean = block_norm(h, **v)
    dh, du = n(10, W), n(10, W).bfloat16()
    clean_b = block_norm_bwd(h, dh, du, **v)
    v["y"] = v["y"].clone()
    v["y"][4, 7] = bad
    out, u = block_norm(h, **v)
    rest = [i for i in range(10) if i != 4]
    assert torch.equal(out[rest], clean[0][rest]) and torch.equal(u[rest], clean[1][rest])
    assert out[4].isnan().any()
    got = block_norm_bwd(h, dh, du, **v)
    assert torch.equal(got[0], clean_b[0])            # the stream's gradient does not see y
    assert torch.equal(got[1][rest], clean_b[1][rest]) and got[1][4].isnan().any()


@pytest.mark.parametrize("gate", ["channel", "token", "full"])
@pytest.mark.parametrize("W", [200, 1800])
def test_gradient_of_y_without_a_norm_does_not_see_y(gate, W):
    h, v, n = draw(10, W, torch.float32, gate, post=False)
    dh, du = n(10, W), n(10, W).bfloat16()
    clean = block_norm_bwd(h, dh, du, **v)
    v["y"] = v["y"].clone()
    v["y"][4, 7], v["y"][5, 8] = float("inf"), float("nan")
    got = block_norm_bwd(h, dh, du, **v)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])


def test_repeats_bit_for_bit():
    h, v, n = draw(3001, 1160, torch.bfloat16)
    dh, du = n(3001, 1160).bfloat16(), n(3001, 1160).bfloat16()
    first = block_norm(h, **v) + block_norm_bwd(h, dh, du, **v)
    for _ in range(3):
        again = block_norm(h, **v) + block_norm_bwd(h, dh, du, **v)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_graph_replays_and_streams():
    h, v, n = draw(300, 1160, torch.float32, gate="token")
    dh, du = n(300, 1160), n(300, 1160).bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block_norm(h, **v)
        block_norm_bwd(h, dh, du, **v)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, u = block_norm(h, **v)
        grads = block_norm_bwd(out, dh, u, **v)
    for i in range(3):
        h.add_(0.25)
        du.mul_(1.5)
        g.replay()
        torch.cuda.synchronize()
        want_out, want_u = block_norm(h, **v)
        want = block_norm_bwd(want_out, dh, want_u, **v)
        torch.cuda.synchronize()
        assert torch.equal(out, want_out) and torch.equal(u, want_u)
        assert all(torch.equal(a, b) for a, b in zip(grads, want))


def test_leading_dimensions():
    h, v, n = draw(24, 128, torch.float32, gate="token")
    out, u = block_norm(h, **v)
    vv = {k: t.view(2, 12, -1) if t is not None and t.dim() == 2 else t for k, t in v.items()}
    o3, u3 = block_norm(h.view(2, 12, 128), **vv)
    assert torch.equal(o3.view(24, 128), out) and torch.equal(u3.view(24, 128), u)


def test_offsets_past_32_bits():
    """Rows whose bytes lie past 2^32, and whose elements lie past 2^31."""
    T, W = 300_000, 7168
    h = torch.zeros((T, W), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((T, W), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    for r in (h, y):
        r[-3:] = torch.randn((3, W), generator=g, device="cuda").bfloat16()
    w = torch.ones(W, device="cuda")
    out, u = block_norm(h, y, w_post=w, w_pre=w, h_out=h.clone())
    want, want_u = block_norm(h[-3:].clone(), y[-3:].clone(), w_post=w, w_pre=w)
    assert torch.equal(out[-3:], want) and torch.equal(u[-3:], want_u)
    assert not out[:-3].any()
    dres, dy, _, dw_post, dw_pre = block_norm_bwd(out, out, u, y, w_post=w, w_pre=w)
    ref = block_norm_bwd(want, want, want_u, y[-3:].clone(), w_post=w, w_pre=w)
    assert torch.equal(dres[-3:], ref[0]) and torch.equal(dy[-3:], ref[1])
    assert not dres[:-3].any() and not dy[:-3].any()
    # the same terms beside zeros, in another order
    for a, b in ((dw_post, ref[3]), (dw_pre, ref[4])):
        assert (a - b).abs().max() <= 8 * E * 3 * b.abs().max()
