"""moonep_orthogonalize of gradients of one token, most of whose norm a few
rows hold, at the precision that the header states."""
import pytest
import torch

from grouped_gemm_moonep_amd import MUON_COEFFS, orthogonalize
from gpu_util import log

pytestmark = pytest.mark.gpu

FIVE = [MUON_COEFFS] * 5


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


# Before the rounding to bf16.  Where a singular value is one, an error e of the first m x m
# matrix reaches the result 1.1e3 times larger, one of the first step's T = R A 6.8e3 times,
# 1.7e3 and 4e2 those of the next two, and an error of each P, or of the last product, 485 times.
# An error is the roundings of three matrices to 22 bits (each 0.6 units of 2^-24) and of N
# additions, four per matrix instruction of 16 values and three of those per 16: 0.75 K for
# a chain over K values, 120 + K / 160 in two sums.  An addition is off by 0.29 units (uniform
# within half a unit of a value below one), so by sqrt(N / 12) together: in units, for K =
# 2048, 6.8e3 * 3.5, 1.7e3 * 11.4, 4e2 * 11.4 and 485 * 2.2 * 11.4, in all 3.3e4 units
# or 2e-3 as the standard deviation for a norm in one or two rows; K = 300: 1.6e-3.  One and a
# half times the first is allowed.
BEFORE = 3e-3


@pytest.mark.parametrize("size,seed", [((180, 300, 310), 301), ((60, 1010, 1025), 1010),
                                       ((32, 2048, 7168), 4), ((6, 7168, 2048), 5)], ids=str)
def test_one_token_whose_norm_few_rows_hold(size, seed):
    n, rows, cols = size
    r = torch.Generator(device="cuda").manual_seed(seed)
    g = torch.empty(size, device="cuda")
    for i in range(n):
        scale = torch.exp(torch.randn((rows,), generator=r, device="cuda"))
        a = torch.randn((1, rows), generator=r, device="cuda")
        g[i] = (a * scale).t() @ (1e-3 * torch.randn((1, cols), generator=r, device="cuda"))
    g = g.bfloat16()
    out = orthogonalize(g)
    worst = before = 0.0
    for i in range(n):
        want = reference(g[i:i + 1])
        norm = torch.linalg.matrix_norm(want)
        rel = torch.linalg.matrix_norm(out[i:i + 1].double() - want) / norm
        # the rounding's square, of 93000 values or more, is within 3% of its mean
        rest = rel ** 2 - 1.03 * (rounding(want) / norm) ** 2
        worst, before = max(worst, rel.item()), max(before, rest.item())
    log(f"ortho {size} of one token: worst {worst:.2e}, "
        f"before the rounding {max(before, 0) ** 0.5:.2e}")
    assert before <= BEFORE ** 2


@pytest.mark.parametrize("size,seed", [((200, 64, 100), 6), ((200, 203, 214), 1), ((60, 487, 1081), 2),
                                       ((86, 900, 1933), 3), ((16, 2048, 7168), 5)], ids=str)
def test_one_token_whose_norm_two_rows_hold(size, seed):
    """Two rows a hundred times the others: the root mean square within the standard deviation
    counted above (1.6e-3 at the shorter sides below 2048, where it is 2e-3), none at three
    times it."""
    n, rows, cols = size
    r = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randn((n, rows, 1), generator=r, device="cuda")
    a[:, 2:] *= 1e-2
    g = torch.stack([a[i] @ (1e-3 * torch.randn((1, cols), generator=r, device="cuda"))
                     for i in range(n)]).bfloat16()
    out = orthogonalize(g)
    before = []
    for i in range(n):
        want = reference(g[i:i + 1])
        norm = torch.linalg.matrix_norm(want)
        rel = torch.linalg.matrix_norm(out[i:i + 1].double() - want) / norm
        before.append(max((rel ** 2 - (rounding(want) / norm) ** 2).item(), 0.0))
    rms, worst = (sum(before) / n) ** 0.5, max(before) ** 0.5
    log(f"ortho {size} of one token, two rows: rms {rms:.2e}, worst {worst:.2e} before the rounding")
    deviation = 2e-3 if min(rows, cols) >= 2048 else 1.6e-3
    assert rms <= deviation and worst <= 3 * deviation
