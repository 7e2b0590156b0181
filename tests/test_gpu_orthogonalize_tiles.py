"""moonep_orthogonalize in every tile that its products can take, with full
and low ranks at the precision that the header states."""
import pytest
import torch

from grouped_gemm_moonep_amd import MUON_COEFFS, _abi, orthogonalize
from gpu_util import log

FIVE = [MUON_COEFFS] * 5

SIZES = [(1, 1024, 2048), (1, 290, 700), (5, 509, 1283), (24, 290, 700), (40, 250, 272),
         (1, 2048, 7168), (1, 7168, 2048), (4, 1024, 2048), (4, 1021, 1500), (3, 1500, 1283),
         (2, 2048, 2048), (9, 1021, 1030), (180, 300, 310),
         (26, 1010, 1025), (8, 2100, 1990), (53, 999, 1024)]

TILES = {_abi.ORTHO_FIRST: {_abi.TILE_64, _abi.TILE_128_DEEP, _abi.TILE_128, _abi.TILE_128X256},
         _abi.ORTHO_R: {_abi.TILE_64, _abi.TILE_128_DEEP, _abi.TILE_128, _abi.TILE_256},
         _abi.ORTHO_TP: {_abi.TILE_64, _abi.TILE_128_DEEP, _abi.TILE_128, _abi.TILE_256},
         _abi.ORTHO_A: {_abi.TILE_64, _abi.TILE_128_DEEP, _abi.TILE_128, _abi.TILE_256},
         _abi.ORTHO_LAST: {_abi.TILE_64, _abi.TILE_128_DEEP, _abi.TILE_256}}


def tile(size, product):
    return _abi.lib().moonep_orthogonalize_tile(*size, product)


@pytest.mark.parametrize("product", _abi.ORTHO_PRODUCTS)
def test_the_sizes_take_every_tile(product):
    """Each among sizes whose edges end inside a tile."""
    assert {tile(s, product) for s in SIZES} == TILES[product]
    for t in TILES[product]:
        assert any(tile(s, product) == t and min(s[1:]) % 32 for s in SIZES), t


def test_tiles_of_other_sizes_stay_in_range():
    for n in (1, 2, 3, 7, 30, 200, 3000):
        for rows in (1, 63, 64, 129, 500, 1000, 2048, 7000):
            for cols in (1, 65, 300, 2000, 7168):
                for product in _abi.ORTHO_PRODUCTS:
                    assert tile((n, rows, cols), product) in TILES[product]
    for bad in ((0, 8, 8, 0), (1, 0, 8, 0), (1, 65537, 8, 0), (1, 8, 8, 5), (1, 8, 8, -1)):
        assert _abi.lib().moonep_orthogonalize_tile(*bad) == -1


def reference(g):
    """The steps in float64 on the device."""
    x = g.double()
    x = x / (torch.linalg.matrix_norm(x, keepdim=True) + 1e-7)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    for a, b, c in FIVE:
        m = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * m + c * torch.bmm(m, m), x)
    return x.transpose(1, 2) if tall else x


def rounding(want):
    """Norm that rounding `want` to bf16 leaves: errors uniform over half a step either way."""
    half = torch.ldexp(torch.ones_like(want), torch.frexp(want).exponent - 9)
    return torch.linalg.matrix_norm(torch.where(want == 0, 0.0, half)) / 3 ** 0.5


def gradients(size, ranks, seed):
    """Matrix i is A^T B of ranks[i % len] tokens, with rows of unequal size; None: of full rank."""
    n, rows, cols = size
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(size, device="cuda")
    for i in range(n):
        t = ranks[i % len(ranks)]
        if t is None:
            out[i] = torch.randn((rows, cols), generator=g, device="cuda")
            continue
        scale = torch.exp(torch.randn((rows,), generator=g, device="cuda"))
        a = torch.randn((t, rows), generator=g, device="cuda") * scale
        out[i] = a.t() @ (1e-3 * torch.randn((t, cols), generator=g, device="cuda"))
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_precision_in_every_tile(size, dtype):
    kinds = [None, 1, 4]
    for shift in range(3 if size[0] < 3 else 1):
        ranks = kinds[shift:] + kinds[:shift]
        g = gradients(size, ranks, 100 * shift + size[1]).to(dtype)
        out = orthogonalize(g)
        again = orthogonalize(g)
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))
        want = reference(g)
        norm = torch.linalg.matrix_norm(want)
        err = torch.linalg.matrix_norm(out.double() - want)
        log(f"ortho {size} {dtype} ranks {ranks[:size[0]]}: worst {(err / norm).max().item():.3e}, "
            f"rounding alone {(rounding(want) / norm).max().item():.3e}")
        # At full rank nothing but the rounding to bf16 (its square within 3% of its mean over
        # 68000 and more entries), and before it 10^-5, for which 10^-4 is allowed.
        full = torch.tensor([ranks[i % 3] is None for i in range(size[0])], device="cuda")
        tol = torch.sqrt(1.03 * rounding(want) ** 2 + (1e-4 * norm) ** 2)
        assert (err <= tol)[full].all(), (err / tol)[full].max()
        # At low rank up to 3 10^-3 before it: test_gpu_orthogonalize_precision.py counts the
        # roundings for rank one (a higher rank spreads them over its directions).
        tol = torch.sqrt(1.03 * rounding(want) ** 2 + (3e-3 * norm) ** 2)
        assert (err <= tol)[~full].all(), (err / norm)[~full].max()
