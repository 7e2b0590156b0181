"""shared_ffn and shared_ffn_bwd at sizes that take every tile and split of
every product, against the oracle (the checks and bounds of
test_gpu_shared_ffn), and every kind of weight gradient's addition."""
import pytest

from shared_ffn_cases import CASES
from test_gpu_shared_ffn import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,Hp", CASES)
def test_every_tile(T, H, Hp):
    check(T, H, Hp, act="gelu_tanh" if T % 2 else "silu", with_add=Hp % 128 == 0, seed=T)


# weight gradients of the small tiles, whole and in splits, of 128- and 256-row large tiles and splits
@pytest.mark.parametrize("T,H,Hp", [(40, 64, 64), (900, 128, 192), (300, 4160, 64), (269, 11328, 64),
                                    (6000, 1088, 512)])
def test_adding_to_fp32(T, H, Hp):
    check(T, H, Hp, f32=True, forward=False, seed=T)
