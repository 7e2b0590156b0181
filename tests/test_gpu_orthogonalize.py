"""moonep_orthogonalize on the GPU against the oracle's Newton-Schulz
iteration in 64 bits: every kernel variant's sizes, both types and
orientations, low ranks, zero, tiny, huge, infinite and NaN matrices, step
coefficients, workspaces, streams, graph replays."""
import numpy as np
import pytest
import torch

from grouped_gemm_moonep_amd import (MUON_COEFFS, MoonepError, orthogonalize,
                                     orthogonalize_workspace)
from gpu_util import log
from oracle import training as T

pytestmark = pytest.mark.gpu

FIVE = [MUON_COEFFS] * 5

# bf16 values are off by at most 2^-8 of themselves.  Before that rounding: a
# relative error e in the first m x m matrix reaches the result, where a
# singular value near one stands beside zeros, as (sum over steps i of 2.74
# a^(5-i) w_i) e, with w_1 = 1, w_(i+1) = 2.4 w_i + 24: under 10^4 e.  e is 2^-24
# times at most four (two roundings to 22 and 24 bits and those of a sum).
TOL = 2.0 ** -8 + 4e4 * 2.0 ** -24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def reference(g, coeffs, eps=1e-7):
    """The oracle's steps on all matrices at once, in float64 on the device."""
    x = g.double()
    x = x / (torch.linalg.matrix_norm(x, keepdim=True) + eps)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    for a, b, c in coeffs:
        m = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * m + c * torch.bmm(m, m), x)
    return x.transpose(1, 2) if tall else x


def check(g, coeffs=FIVE, eps=1e-7, what="", **kw):
    out = orthogonalize(g, steps=len(coeffs), coeffs=coeffs, eps=eps, **kw)
    assert out.dtype == torch.bfloat16 and out.shape == g.shape
    want = reference(g, coeffs, eps)
    norm = torch.linalg.matrix_norm(want)
    err = torch.linalg.matrix_norm(out.double() - want)
    rel = (err / norm.clamp_min(1e-30))
    log(f"ortho {tuple(g.shape)} {what}: worst relative error {rel.max().item():.2e}")
    assert torch.isfinite(out).all() and (err <= TOL * norm).all(), rel.max()
    return out


def test_reference_is_the_oracle():
    g = torch.randn((2, 9, 5), generator=gen(0), device="cuda")
    want = np.stack([T.orthogonalize(m, FIVE) for m in g.cpu().numpy()])
    assert np.allclose(reference(g, FIVE).cpu().numpy(), want, atol=1e-12)


# one tile per matrix, its border, several tiles with few and with many workgroups, and more
# matrices than one group takes
SIZES = [(1, 1, 1), (1, 1, 7), (3, 5, 3), (2, 33, 31), (2, 64, 130), (1, 127, 300), (2, 128, 128),
         (1, 128, 129), (1, 129, 128), (1, 129, 131), (2, 200, 515), (3, 257, 256), (1, 512, 513),
         (1, 300, 1000), (90, 130, 140), (40, 250, 272), (520, 256, 256), (180, 300, 310),
         (520, 200, 250), (2100, 8, 12), (4, 16, 2048)]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_matches_reference(size):
    n, rows, cols = size
    g = torch.randn((n, rows, cols), generator=gen(rows * 7 + cols), device="cuda")
    check(g, what="fp32")
    if n <= 4:
        check(g.transpose(1, 2).contiguous(), what="transposed")
        check(g.bfloat16(), what="bf16")


# 256-wide tiles, some of them in quarters, with odd edges; the 128 x 256 ones of the first product
@pytest.mark.parametrize("size", [(26, 1010, 1025), (8, 2100, 1990), (53, 999, 1024)], ids=str)
def test_large_tiles(size):
    n, rows, cols = size
    r = gen(n)
    g = torch.randn(size, generator=r, device="cuda")
    g[1] = torch.randn((rows, 2), generator=r, device="cuda") @ g[1, :2]
    check(g, what="large tiles")


@pytest.mark.parametrize("size", [(1, 65536, 8), (2, 8, 65536), (1, 40, 65533)], ids=str)
def test_longest_sides(size):
    check(torch.randn(size, generator=gen(1), device="cuda"), what="longest sides")


# One entry per row, in columns of its own: its size is a singular value, so the result has the
# same pattern and every entry goes through the steps alone.  Nearly as many elements as the call
# takes, in both orientations; offsets pass 2^31 bytes in g, X_0 and the workspace.
@pytest.mark.parametrize("transposed", [False, True])
def test_largest_matrix(transposed):
    m, n = 16384, 32760
    r = gen(3)
    col = torch.randperm(n, generator=r, device="cuda")[:m]
    row = torch.arange(m, device="cuda")
    value = torch.randn((m,), generator=r, device="cuda")
    g = torch.zeros((n, m) if transposed else (m, n), device="cuda")
    at = (col, row) if transposed else (row, col)
    g[at] = value
    out = orthogonalize(g)
    x = value.double() / (torch.linalg.vector_norm(value.double()) + 1e-7)
    for a, b, c in FIVE:
        x = x * (a + b * x ** 2 + c * x ** 4)
    got = out[at].double()
    assert ((got - x).abs() <= 2.0 ** -8 * x.abs() + 4e4 * 2.0 ** -24).all()
    out[at] = 0
    assert not out.any()


def test_no_matrices():
    assert orthogonalize(torch.empty((0, 5, 7), device="cuda")).shape == (0, 5, 7)


@pytest.mark.parametrize("tokens", [1, 2, 5, 40])
@pytest.mark.parametrize("rows,cols", [(64, 96), (200, 515), (509, 1283)])
def test_low_rank_gradients(tokens, rows, cols):
    """A^T B of few tokens, rows of unequal size: most singular values are
    zero, or the rounding of the gradient itself."""
    g = gen(tokens)
    a = torch.randn((tokens, rows), generator=g, device="cuda")
    a *= torch.exp(torch.randn((rows,), generator=g, device="cuda"))
    b = 1e-3 * torch.randn((tokens, cols), generator=g, device="cuda")
    m = (a.t() @ b)[None].contiguous()
    check(m, what=f"rank {tokens}")
    check(m.bfloat16(), what=f"rank {tokens} bf16")


# Rows of very unequal size, where single entries of the first matrices decide.
# Rounding to bf16 leaves at most 2^-8 / sqrt(3) of the norm (errors uniform over
# half a step); the roundings before it are independent per entry, so 10^4 times
# two of 2^-24 / sqrt(3) rather than four times 2^-24: 2.4e-3 together.
@pytest.mark.parametrize("n,rows,cols,tokens,spread", [(1, 848, 1152, 1, 1), (1, 500, 1100, 4, 1),
                                                       (2, 114, 111, 4, 0), (1, 1000, 1100, 2, 1),
                                                       (20, 260, 600, 1, 1)])
def test_low_rank_gradients_of_unequal_rows(n, rows, cols, tokens, spread):
    r = gen(tokens)
    scale = torch.exp(spread * torch.randn((rows,), generator=r, device="cuda"))
    g = torch.stack([(torch.randn((tokens, rows), generator=r, device="cuda") * scale).t() @
                     (1e-3 * torch.randn((tokens, cols), generator=r, device="cuda"))
                     for _ in range(n)]).to(torch.bfloat16)
    want = reference(g, FIVE)
    rel = (torch.linalg.matrix_norm(orthogonalize(g).double() - want) /
           torch.linalg.matrix_norm(want))
    log(f"ortho {tuple(g.shape)} of {tokens} tokens, unequal rows: {rel.max().item():.2e}")
    assert (rel <= 2.4e-3).all(), rel


def test_headline_gradient():
    g = torch.randn((2, 7168, 2048), generator=gen(1), device="cuda")
    g[1, :, 300:] *= 1e-4
    check(g, what="headline")


def test_sizes_of_values():
    """Gradients far below and above one, whose squares leave fp32's range."""
    base = torch.randn((1, 60, 100), generator=gen(2), device="cuda")
    want = check(base, eps=1e-30)
    for scale in (1e-25, 1e-12, 1e12, 1e25):
        got = check(base * scale, eps=1e-30, what=f"times {scale:g}")
        assert (got.float() - want.float()).abs().max() < 2 * 2.0 ** -8
    small = check(base * 1e-9, eps=1e-7)                 # eps counts here
    assert not torch.equal(small, want)


@pytest.mark.parametrize("scale", [1e-8, 1e-13, 1e-20, 1e-30])
def test_gradients_far_below_eps(scale):
    """The result is then about the gains' product times G / eps, small but not lost."""
    g = torch.randn((3, 60, 100), generator=gen(2), device="cuda") * scale
    g[1] *= 1e3
    check(g, what=f"times {scale:g}, eps 1e-7")
    check(g.transpose(1, 2).contiguous().bfloat16(), what=f"times {scale:g}, eps 1e-7")


def test_zero_and_bad_matrices_stay_by_themselves():
    for shape in ((5, 40, 60), (5, 140, 200)):
        g = torch.randn(shape, generator=gen(3), device="cuda")
        ref = orthogonalize(g)
        g[1] = 0
        g[2, 3, 4] = float("nan")
        g[3, 0, 0] = float("inf")
        out = orthogonalize(g)
        assert not out[1].any()
        assert torch.isnan(out[2]).all() and not torch.isfinite(out[3]).any()
        for i in (0, 4):
            assert torch.equal(out[i].view(torch.int16), ref[i].view(torch.int16))


@pytest.mark.parametrize("coeffs", [[MUON_COEFFS], FIVE[:2], [(1.5, -0.5, 0.0)] * 8,
                                    [(4.0, -6.5, 3.2), (3.0, -3.5, 1.4), (2.0, -1.5, 0.5)]])
@pytest.mark.parametrize("rows,cols", [(70, 50), (300, 260)])
def test_step_coefficients(coeffs, rows, cols):
    check(torch.randn((2, rows, cols), generator=gen(4), device="cuda"), coeffs=coeffs,
          what=f"{len(coeffs)} steps")


def test_two_dimensions_given_buffers_and_unaligned_storage():
    store = torch.randn(1 + 3 * 45 * 77, generator=gen(5), device="cuda")
    g = store[1:].view(3, 45, 77)                         # rows on 4 bytes
    ws = orthogonalize_workspace(3, 45, 77)
    obuf = torch.full((1 + g.numel(),), 7.0, dtype=torch.bfloat16, device="cuda")
    out = obuf[1:].view(g.shape)
    assert orthogonalize(g, out=out, ws=ws) is out
    assert obuf[0] == 7
    want = orthogonalize(g.clone())
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    one = orthogonalize(g[1].contiguous())
    assert one.shape == (45, 77)
    assert torch.equal(one.view(torch.int16), want[1].view(torch.int16))
    assert orthogonalize(torch.empty((0, 4, 5), device="cuda")).shape == (0, 4, 5)


def test_streams_with_their_own_workspaces():
    gs = [torch.randn((6, 200, 300), generator=gen(i), device="cuda") for i in range(3)]
    want = [orthogonalize(g) for g in gs]
    torch.cuda.synchronize()
    got = [None] * 3
    streams = [torch.cuda.Stream() for _ in gs]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            got[i] = orthogonalize(gs[i])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("size", [(3, 60, 100), (5, 260, 150), (520, 200, 256)], ids=str)
def test_graph_replays_equal_eager(size):
    g = torch.empty(size, device="cuda")
    ws = orthogonalize_workspace(*size)
    out = torch.empty(size, dtype=torch.bfloat16, device="cuda")
    ins = [torch.randn(size, generator=gen(i), device="cuda") for i in range(3)]
    refs = [orthogonalize(v) for v in ins]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.copy_(ins[0])
        orthogonalize(g, out=out, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        orthogonalize(g, out=out, ws=ws)
    for rep in range(2):
        for v, r in zip(ins, refs):
            g.copy_(v)
            out.fill_(3)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out.view(torch.int16), r.view(torch.int16))
            ws.fill_(0xFF)                               # nothing is kept in the workspace
            torch.cuda.synchronize()
    del graph


def test_refusals():
    g = torch.zeros((2, 8, 8), device="cuda")
    ws = orthogonalize_workspace(2, 8, 8)
    for bad, kind in [(dict(out=g), TypeError), (dict(out=g.bfloat16()[:1]), ValueError),
                      (dict(ws=ws[:-1]), MoonepError), (dict(ws=ws.float()), TypeError),
                      (dict(ws=ws[1:]), MoonepError),
                      (dict(out=g.view(torch.bfloat16).view(-1)[:128].view(2, 8, 8)), ValueError),
                      (dict(steps=0), MoonepError), (dict(eps=0.0), MoonepError),
                      (dict(coeffs=(-1.0, 0.0, 0.0)), MoonepError),
                      (dict(steps=7), MoonepError)]:
        with pytest.raises(kind):
            orthogonalize(g, **bad)
    with pytest.raises(ValueError, match="contiguous"):
        orthogonalize(g.transpose(1, 2)[:, :, :4])
