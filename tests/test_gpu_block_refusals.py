"""What the binding of block_norm and shared_ffn refuses of device tensors (types, shapes, strides,
devices, overlaps, workspaces), parts of a backward alone, and two calls at once."""
import pytest
import torch

import grouped_gemm_moonep_amd as moonep
from grouped_gemm_moonep_amd import block_norm, block_norm_bwd, shared_ffn, shared_ffn_bwd

pytestmark = pytest.mark.gpu


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


def f32(*shape):
    return torch.zeros(shape, device="cuda")


@pytest.mark.parametrize("name,make,error", [
    ("h", lambda: f32(6, 64).double(), TypeError), ("h", lambda: f32(64, 6).t(), ValueError),
    ("y", lambda: f32(6, 64), TypeError), ("y", lambda: bf(5, 64), ValueError),
    ("y", lambda: bf(64, 6).t(), ValueError), ("y", lambda: bf(6, 64).cpu(), ValueError),
    ("y", lambda: None, ValueError), ("y2", lambda: bf(6, 32), ValueError),
    ("w_post", lambda: bf(64), TypeError), ("w_pre", lambda: f32(32), ValueError),
    ("gate", lambda: f32(6), ValueError), ("gate", lambda: f32(6, 64), ValueError),
    ("gate", lambda: bf(64), ValueError), ("gate", lambda: f32(6, 1).half(), TypeError),
    ("eps", lambda: 0.0, moonep.MoonepError), ("scale", lambda: float("nan"), moonep.MoonepError),
    ("u", lambda: f32(6, 64), TypeError), ("h_out", lambda: f32(6, 32), ValueError),
    ("h_out", lambda: bf(6, 64), TypeError)])
def test_norm_arguments(name, make, error):
    a = dict(h=f32(6, 64), y=bf(6, 64), w_post=f32(64), w_pre=f32(64))
    a[name] = make()
    with pytest.raises(error):
        block_norm(**a)
    if name not in ("u", "h_out"):
        with pytest.raises(error):
            block_norm_bwd(dh=f32(6, 64), du=bf(6, 64), **a)


def test_norm_overlaps():
    store = torch.zeros(1 << 16, device="cuda")
    part = lambda at: store[at:at + 384].view(6, 64)
    half = lambda at: store.view(torch.bfloat16)[at:at + 384].view(6, 64)
    h = part(0)
    a = dict(y=half(768), w_post=f32(64), w_pre=f32(64))         # y is store[384:576]
    for bad, what in ((dict(h_out=part(64)), "h_out must not overlap h"),
                      (dict(h_out=part(512)), "h_out must not overlap y"),
                      (dict(u=half(128)), "u must not overlap h"),
                      (dict(u=half(784)), "u must not overlap y"),
                      (dict(h_out=part(1024), u=half(2112)), "u must not overlap h_out")):
        with pytest.raises(ValueError, match=what):
            block_norm(h, **a, **bad)
    dh, du = part(1024), half(4096)
    for bad, what in ((dict(dres=h), "dres must not overlap h"),
                      (dict(dres=part(1088)), "dres must not overlap dh"),
                      (dict(dy=half(4112)), "dy must not overlap du"),
                      (dict(dres=part(4096), dy=half(8200)), "dy must not overlap dres"),
                      (dict(ws=store.view(torch.uint8)), "ws must not overlap h")):
        with pytest.raises(ValueError, match=what):
            block_norm_bwd(h, dh, du, **a, **bad)
    space = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    for ws in (space[:16], space[8:]):                            # too small; not aligned
        with pytest.raises(moonep.MoonepError):
            block_norm_bwd(h, dh, du, **a, ws=ws)
    assert not store.any()


@pytest.mark.parametrize("name,make,error", [
    ("x", lambda: f32(5, 64), TypeError), ("x", lambda: bf(5, 128), ValueError),
    ("x", lambda: bf(64, 5).t(), ValueError), ("x", lambda: bf(5, 64).cpu(), ValueError),
    ("weights", lambda: [bf(64, 128)] * 2, ValueError),
    ("weights", lambda: [bf(64, 128)] * 2 + [bf(128, 64)], ValueError),
    ("weights", lambda: [bf(64, 128)] * 2 + [f32(64, 128)], TypeError),
    ("weights", lambda: [bf(64, 128)] * 2 + [bf(128, 64).t()], ValueError),
    ("weights", lambda: [bf(64, 96)] * 3, moonep.MoonepError),
    ("act", lambda: "gelu", ValueError), ("ws", lambda: f32(1 << 20), TypeError),
    ("ws", lambda: torch.zeros(256, dtype=torch.uint8, device="cuda"), moonep.MoonepError),
    ("ws", lambda: torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")[16:], moonep.MoonepError)])
def test_ffn_arguments(name, make, error):
    a = dict(x=bf(5, 64), weights=[bf(64, 128) for _ in range(3)])
    a[name] = make()
    with pytest.raises(error):
        shared_ffn(**a)
    with pytest.raises(error):
        shared_ffn_bwd(dy=bf(5, 64), **a)


def test_ffn_overlaps():
    x, dy, w = bf(5, 64), bf(5, 64), [bf(64, 128) for _ in range(3)]
    g = [bf(64, 128) for _ in range(3)]
    rows = bf(8, 64)
    for bad, what in ((dict(out=x), "out must not overlap x"),
                      (dict(out=w[2].view(-1)[:320].view(5, 64)), "out must not overlap down"),
                      (dict(out=rows[1:6], add=rows[:5]), "out must not overlap add")):
        with pytest.raises(ValueError, match=what):
            shared_ffn(x, w, **bad)
    for bad, what in ((dict(dx=dy), "dx must not overlap dy"), (dict(dx=x), "dx must not overlap x"),
                      (dict(dw=[g[0], g[0], g[1]]), r"dw\[1\] must not overlap dw\[0\]"),
                      (dict(dw=[g[0], g[1], w[0]]), r"dw\[2\] must not overlap gate"),
                      (dict(dw=g, need_dw=False), "need_dw"), (dict(dx=rows[:5], need_dx=False), "need_dx"),
                      (dict(dw=g[:2]), "three gradients")):
        with pytest.raises(ValueError, match=what):
            shared_ffn_bwd(x, dy, w, **bad)
    with pytest.raises(TypeError):
        shared_ffn_bwd(x, dy, w, dw=[g[0], g[1], f32(64, 128)])


def inputs(T, H, Hp):
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    return n(T, H).bfloat16(), n(T, H).bfloat16(), [(n(H, Hp) * H ** -0.5).bfloat16() for _ in range(3)]


@pytest.mark.parametrize("T,H,Hp", [(3000, 2048, 1408), (8168, 1024, 2048), (4100, 4096, 4160),
                                    (1100, 2048, 1024), (90, 4096, 64)])
def test_parts_of_the_backward_alone(T, H, Hp):
    """dX and the weight gradients, in one launch where their tiles are alike, against each alone:
    the same sums, bit for bit, in bf16 and added to fp32."""
    x, dy, w = inputs(T, H, Hp)
    dx, dw = shared_ffn_bwd(x, dy, w)
    only, none = shared_ffn_bwd(x, dy, w, need_dw=False)
    gone, alone = shared_ffn_bwd(x, dy, w, need_dx=False)
    assert none is None and gone is None
    assert torch.equal(dx, only) and all(torch.equal(a, b) for a, b in zip(dw, alone))
    one, two = ([f32(H, Hp) for _ in range(3)] for _ in range(2))
    also, _ = shared_ffn_bwd(x, dy, w, dw=one)
    shared_ffn_bwd(x, dy, w, need_dx=False, dw=two)
    assert torch.equal(also, dx) and all(torch.equal(a, b) for a, b in zip(one, two))
    assert all(torch.equal(a.bfloat16(), b) for a, b in zip(one, dw))


def test_two_calls_at_once():
    """Two streams run different sizes of every call side by side: the results are those of either alone."""
    def work(T, H, Hp):
        x, dy, w = inputs(T, H, Hp)
        wn = torch.linspace(0.5, 1.5, H, device="cuda")

        def run():
            z = shared_ffn(x, w, add=dy)
            dx, dw = shared_ffn_bwd(x, dy, w)
            h, u = block_norm(x.float(), z, gate=wn, w_post=wn, w_pre=wn)
            return (z, dx, *dw, h, u, *block_norm_bwd(h, h, u, z, gate=wn, w_post=wn, w_pre=wn)[:5])
        return run
    runs = [work(300, 1024, 512), work(17, 2048, 192)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [[], []]
    for _ in range(4):
        for i, (s, r) in enumerate(zip(streams, runs)):
            with torch.cuda.stream(s):
                got[i].append(r())
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        for g in gs:
            assert all(torch.equal(a, b) for a, b in zip(w, g))
