"""shared_ffn and shared_ffn_bwd on the GPU against the oracle in float64:
token counts from one across every tile's edge, hidden sizes that are odd
multiples of 64, both activations, with and without what is added, both types
of weight gradients, graphs, streams, repeats, untouched surroundings.

Tolerances count roundings, e = 2^-24 and b = 2^-8 (half a step of bf16): a
product of K terms summed in fp32 is off by at most (K + 8) e of its terms'
magnitudes, Z, dG and dU by b of their value more, and a bf16 result by b of
its own; every bound below is the sum of these through the formulas."""
import numpy as np
import pytest
import torch

from gpu_util import log
from grouped_gemm_moonep_amd import (shared_ffn, shared_ffn_bwd, shared_ffn_bwd_workspace,
                                     shared_ffn_workspace)
from oracle import block as B

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
HALF = torch.finfo(torch.bfloat16).eps / 2
ACT_E = 64 * E            # exponential, reciprocal and products of an activation, of its parts


def draw(T, H, Hp, seed=0, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = n(T, H).bfloat16()
    w = tuple((n(H, Hp) * (scale / s ** 0.5)).bfloat16() for s in (H, H, Hp))
    return x, w, n(T, H).bfloat16(), n(T, H).bfloat16()


def wide(t):
    return t.double().cpu().numpy()


def within(got, want, err, what):
    got = wide(got)
    assert got.shape == want.shape, what
    worst = float((np.abs(got - want) / (err + 1e-30)).max()) if got.size else 0.0
    log(f"{what}: worst error / bound {worst:.3f}")
    assert worst <= 1.0, f"{what}: {worst:.3f} of its bound"


class Exact:
    """The values of a case and how far each may be off."""

    def __init__(self, x, w, act):
        self.x, self.w, self.act = wide(x), [wide(t) for t in w], act
        ax, aw = np.abs(self.x), [np.abs(t) for t in self.w]
        H, Hp = self.w[0].shape
        self.g, self.u = self.x @ self.w[0], self.x @ self.w[1]
        self.eg, self.eu = (H + 8) * E * (ax @ aw[0]), (H + 8) * E * (ax @ aw[1])
        self.f, self.df = B.act(self.g, act)
        # |f'| <= 1.2 and |f''| <= 1.2 for both activations
        self.ef = 1.2 * self.eg + ACT_E * (np.abs(self.g) + 1e-3)
        self.edf = 1.2 * self.eg + ACT_E * (np.abs(self.g) + 1)
        self.z = self.f * self.u
        ez = self.ef * np.abs(self.u) + (np.abs(self.f) + self.ef) * self.eu + 2 * E * np.abs(self.z)
        self.ez = ez + HALF * (np.abs(self.z) + ez)
        self.aw, self.Hp = aw, Hp

    def forward(self, add):
        y = self.z @ self.w[2].T
        mag = np.abs(self.z) @ self.aw[2].T
        e = self.ez @ self.aw[2].T + (self.Hp + 8) * E * mag
        if add is not None:
            y = y + wide(add)
            e = e + 2 * E * np.abs(wide(add))
        return y, e + HALF * (np.abs(y) + e)

    def backward(self, dy):
        d = wide(dy)
        T, H = d.shape
        dz = d @ self.w[2]
        edz = (H + 8) * E * (np.abs(d) @ self.aw[2])
        dg, du = dz * self.u * self.df, dz * self.f
        edu = edz * (np.abs(self.f) + self.ef) + np.abs(dz) * self.ef + 2 * E * np.abs(du)
        au, adf = np.abs(self.u) + self.eu, np.abs(self.df) + self.edf
        edg = edz * au * adf + np.abs(dz) * (self.eu * adf + au * self.edf) + 3 * E * np.abs(dg)
        edu, edg = edu + HALF * (np.abs(du) + edu), edg + HALF * (np.abs(dg) + edg)
        dx = dg @ self.w[0].T + du @ self.w[1].T
        ex = (edg + (2 * self.Hp + 8) * E * np.abs(dg)) @ self.aw[0].T + \
            (edu + (2 * self.Hp + 8) * E * np.abs(du)) @ self.aw[1].T
        ax, ad = np.abs(self.x), np.abs(d)
        s = (T + 16) * E
        dw = (self.x.T @ dg, self.x.T @ du, d.T @ self.z)
        ew = (ax.T @ (edg + s * np.abs(dg)), ax.T @ (edu + s * np.abs(du)),
              ad.T @ (self.ez + s * np.abs(self.z)))
        return dx, ex + HALF * (np.abs(dx) + ex), dw, ew


def check(T, H, Hp, act="silu", with_add=True, backward=True, forward=True, f32=False, seed=0):
    what = f"shared_ffn T={T} H={H} Hp={Hp} {act}"
    log(what)
    x, w, add, dy = draw(T, H, Hp, seed)
    x0, w0, dy0 = x.clone(), [t.clone() for t in w], dy.clone()
    ex = Exact(x, w, act)
    if forward:
        y = shared_ffn(x, w, act=act, add=add if with_add else None)
        want, err = ex.forward(add if with_add else None)
        within(y, want, err, what + " y")
        # the worst case over all terms is far from what independent roundings
        # leave: two of them at most, and rarely both at their largest
        assert np.linalg.norm(wide(y) - want) <= HALF * np.linalg.norm(want)
    if backward:
        dw = tuple(torch.full((H, Hp), 0.5, device="cuda") for _ in range(3)) if f32 else None
        dx, dw = shared_ffn_bwd(x, dy, w, act=act, dw=dw)
        want, err, wants, errs = ex.backward(dy)
        within(dx, want, err, what + " dx")
        for got, a, e, name in zip(dw, wants, errs, ("dWg", "dWu", "dWd")):
            if f32:
                within(got, a + 0.5, e + E * (np.abs(a) + 0.5), f"{what} {name} fp32")
            else:
                within(got, a, e + HALF * (np.abs(a) + e), f"{what} {name}")
    assert torch.equal(x, x0) and torch.equal(dy, dy0)
    assert all(torch.equal(a, b) for a, b in zip(w, w0))


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 127, 129, 257])
@pytest.mark.parametrize("H,Hp", [(64, 64), (320, 192), (192, 576)])
def test_few_tokens(T, H, Hp):
    check(T, H, Hp, act="gelu_tanh" if T % 2 else "silu", with_add=T % 3 != 0)


@pytest.mark.parametrize("T,H,Hp", [
    (1, 1984, 1024), (8, 7168, 512), (40, 2048, 1024), (100, 1024, 2048), (300, 1984, 704),
])
def test_split_products(T, H, Hp):
    """Sizes whose products are cut along K."""
    check(T, H, Hp)


@pytest.mark.parametrize("T,H,Hp,act", [
    (4200, 1024, 2112, "silu"),        # 256-row tiles; the last one of 104 rows
    (4060, 1088, 2048, "gelu_tanh"),   # the last one of 220 rows; 64 columns in the last N-tile
    (3000, 512, 1024, "silu"),         # 128-row tiles of the large kind
    (12301, 128, 192, "silu"),         # few columns; a long sum over the tokens in splits
    (2048, 2048, 4096, "gelu_tanh"),   # weight gradients in large tiles
])
def test_large_tiles(T, H, Hp, act):
    check(T, H, Hp, act=act)


@pytest.mark.parametrize("T,H,Hp", [(50, 128, 192), (700, 256, 320), (600, 2048, 4160)])
def test_fp32_weight_gradients_accumulate(T, H, Hp):
    check(T, H, Hp, f32=True, forward=False)


def test_one_activation_value():
    """Activations far to either side: no overflow, and zero gradients where they are flat."""
    for act in ("silu", "gelu_tanh"):
        x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
        w = [torch.zeros((64, 64), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        x[:, 0] = torch.tensor([1e4, -1e4, 3e19, -3e19], device="cuda")
        w[0][0, :] = 1.0                                      # G = x
        x[:, 1] = 1.0
        w[1][1, :] = 1.0                                      # U = 1
        w[2][0, :] = 2.0 ** -6                                # y[:, 0] = mean of Z
        y = shared_ffn(x, w, act=act)
        want = torch.tensor([1e4, 0.0, 3e19, 0.0], device="cuda").bfloat16()
        assert torch.equal(y[:, 0], want) and not y[:, 1:].any()
        dy = torch.zeros_like(x)
        dy[:, 0] = 1.0
        dx, dw = shared_ffn_bwd(x, dy, w, act=act)
        assert torch.isfinite(dx).all() and all(torch.isfinite(t).all() for t in dw)
        assert torch.equal(dx[:, 0], torch.tensor([1.0, 0, 1.0, 0], device="cuda").bfloat16())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("T", [5, 20000])
def test_gradient_far_below_the_activation(act, T):
    """A gate of -1e33 or below: f and f' are 0, whatever g times the inner derivative would be."""
    x = torch.zeros(T, 128, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = -1e17, 1.0
    w = [torch.zeros(128, 256, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    w[0][0], w[1][1], w[2][2] = 1e16, 1.0, 1.0
    dy = torch.ones_like(x)
    assert not shared_ffn(x, w, act=act).any()
    dx, dw = shared_ffn_bwd(x, dy, w, act=act)
    assert not dx.any() and not any(t.any() for t in dw)


def test_bad_values_stay_in_their_token():
    x, w, add, dy = draw(70, 192, 128)
    clean, (cdx, _) = shared_ffn(x, w, add=add), shared_ffn_bwd(x, dy, w)
    for bad in (float("nan"), float("inf")):
        x2 = x.clone()
        x2[37, 5] = bad
        y, (dx, _) = shared_ffn(x2, w, add=add), shared_ffn_bwd(x2, dy, w)
        rest = [i for i in range(70) if i != 37]
        assert torch.equal(y[rest], clean[rest]) and torch.equal(dx[rest], cdx[rest])
        assert y[37].isnan().any()


def test_what_is_asked_for_and_in_place():
    x, w, add, dy = draw(90, 256, 320)
    want = shared_ffn(x, w, add=add)
    a2 = add.clone()
    assert shared_ffn(x, w, add=a2, out=a2) is a2 and torch.equal(a2, want)
    dx, dw = shared_ffn_bwd(x, dy, w)
    only, none = shared_ffn_bwd(x, dy, w, need_dw=False)
    assert none is None and torch.equal(only, dx)
    none, only = shared_ffn_bwd(x, dy, w, need_dx=False)
    assert none is None and all(torch.equal(a, b) for a, b in zip(only, dw))


def test_no_tokens():
    x, w, _, dy = draw(0, 128, 192)
    assert shared_ffn(x, w).shape == (0, 128)
    dx, dw = shared_ffn_bwd(x, dy, w)
    assert dx.shape == (0, 128) and all(not t.any() for t in dw)
    acc = tuple(torch.full((128, 192), 2.0, device="cuda") for _ in range(3))
    shared_ffn_bwd(x, dy, w, dw=acc)
    assert all(bool((t == 2.0).all()) for t in acc)


@pytest.mark.parametrize("T,H,Hp", [(5, 128, 192), (130, 320, 64), (2500, 1088, 1088)])
def test_surroundings_stay(T, H, Hp):
    """Outputs and workspace lie inside larger arrays whose other elements keep their values."""
    x, w, add, dy = draw(T, H, Hp)
    guard = 4096

    def inside(n, dtype):
        t = torch.full((n + 2 * guard,), 7, dtype=dtype, device="cuda")
        return t, t[guard:guard + n]

    kept = []
    def out(shape, dtype=torch.bfloat16):
        t, v = inside(int(np.prod(shape)), dtype)
        kept.append((t, v.numel()))
        return v.view(shape)

    y = shared_ffn(x, w, add=add, out=out((T, H)),
                   ws=out((shared_ffn_workspace(T, H, Hp).numel(),), torch.uint8))
    dx, dw = shared_ffn_bwd(x, dy, w, dx=out((T, H)), dw=[out((H, Hp)) for _ in range(3)],
                            ws=out((shared_ffn_bwd_workspace(T, H, Hp).numel(),), torch.uint8))
    torch.cuda.synchronize()
    for t, n in kept:
        assert bool((t[:guard] == 7).all()) and bool((t[guard + n:] == 7).all())
    assert torch.equal(y, shared_ffn(x, w, add=add))
    dx2, dw2 = shared_ffn_bwd(x, dy, w)
    assert torch.equal(dx, dx2) and all(torch.equal(a, b) for a, b in zip(dw, dw2))


@pytest.mark.parametrize("T,H,Hp", [(8, 1024, 512), (200, 512, 640), (3000, 512, 1024)])
def test_repeats_graphs_and_streams(T, H, Hp):
    x, w, add, dy = draw(T, H, Hp)
    first = (shared_ffn(x, w, add=add), *shared_ffn_bwd(x, dy, w)[1])
    for _ in range(3):
        again = (shared_ffn(x, w, add=add), *shared_ffn_bwd(x, dy, w)[1])
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    ws, wsb = shared_ffn_workspace(T, H, Hp), shared_ffn_bwd_workspace(T, H, Hp)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = shared_ffn(x, w, add=add, ws=ws)
        shared_ffn_bwd(x, dy, w, ws=wsb)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, first[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = shared_ffn(x, w, add=add, ws=ws)
        dx, dw = shared_ffn_bwd(x, y, w, ws=wsb)
    for i in range(3):
        x.mul_(1.25)
        g.replay()
        torch.cuda.synchronize()
        want = shared_ffn(x, w, add=add)
        wdx, wdw = shared_ffn_bwd(x, want, w)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(dx, wdx)
        assert all(torch.equal(a, b) for a, b in zip(dw, wdw))


def test_leading_dimensions():
    x, w, add, dy = draw(24, 128, 64)
    y = shared_ffn(x.view(2, 12, 128), w, add=add.view(2, 12, 128))
    assert torch.equal(y.view(24, 128), shared_ffn(x, w, add=add))
    dx, _ = shared_ffn_bwd(x.view(2, 12, 128), dy.view(2, 12, 128), w)
    assert dx.shape == (2, 12, 128)


def test_gradients_against_differences():
    """Directional differences of the forward itself, in float64 on the host, for what the GPU's
    gradients say."""
    x, w, _, dy = draw(33, 128, 192)
    dx, dw = shared_ffn_bwd(x, dy, w, act="gelu_tanh")
    xs, ws, d = wide(x), [wide(t) for t in w], wide(dy)
    rng = np.random.default_rng(0)
    f = lambda x, w: float((d * B.shared_ffn(x, w, "gelu_tanh")).sum())
    for k, got in enumerate((dx, *dw)):
        v = rng.standard_normal(got.shape)
        move = lambda s: f(xs + s * v if k == 0 else xs,
                           [t + s * v if k == i + 1 else t for i, t in enumerate(ws)])
        diff = (move(1e-5) - move(-1e-5)) / 2e-5
        # roundings of the gradient: at most three of 2^-8 an element, and v is of both signs
        lim = 3 * HALF * np.abs(wide(got) * v).sum()
        assert abs(diff - float((wide(got) * v).sum())) <= lim


def test_offsets_past_32_bits():
    """Tokens whose elements lie past 2^31."""
    T, H, Hp = 34_000, 64 * 1024, 64
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    x[-3:] = torch.randn((3, H), generator=g, device="cuda").bfloat16()
    w = [(torch.randn((H, Hp), generator=g, device="cuda") / 256).bfloat16() for _ in range(3)]
    y = shared_ffn(x, w)
    want, err = Exact(x[-3:], w, "silu").forward(None)
    within(y[-3:], want, err, "last tokens")
    assert not y[:-3].any()
