"""shared_ffn_bwd at sizes that take every form of the launch that computes dX
and the weight gradients together, against the oracle (the checks and bounds of
test_gpu_shared_ffn), the weight gradients written and added to; and of the
weight gradients' own launch, added to gradients that are not zero."""
import pytest
import torch

from grouped_gemm_moonep_amd import shared_ffn_bwd
from shared_ffn_last_cases import ALONE, LAST
from test_gpu_shared_ffn import check, draw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,H,Hp", list(LAST))
def test_one_launch(T, H, Hp, f32):
    check(T, H, Hp, act="gelu_tanh" if T % 2 else "silu", f32=f32, forward=False, seed=T)


@pytest.mark.parametrize("T,H,Hp", list(ALONE))
def test_adding_in_every_tile(T, H, Hp):
    check(T, H, Hp, f32=True, forward=False, seed=T)


@pytest.mark.parametrize("T,H,Hp", list(LAST))
def test_apart_they_are_the_same(T, H, Hp):
    """Each asked for alone, in launches of their own, gives the same bits."""
    x, w, _, dy = draw(T, H, Hp)
    dx, dw = shared_ffn_bwd(x, dy, w)
    assert torch.equal(dx, shared_ffn_bwd(x, dy, w, need_dw=False)[0])
    alone = shared_ffn_bwd(x, dy, w, need_dx=False)[1]
    assert all(torch.equal(a, b) for a, b in zip(dw, alone))
