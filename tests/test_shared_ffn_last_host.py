"""Host-only checks of moonep_shared_ffn_last_tile: what it says of the launch that takes dX and the
weight gradients together, and that the GPU tests' sizes take every form of it."""
import math
import random

import pytest

from grouped_gemm_moonep_amd import _abi
from shared_ffn_last_cases import ALONE, DEEP, LAST


def blocks(T, H, Hp, tile):
    """Workgroups of a small tile's dX and of the weight gradients beside it, each a multiple of the
    eight XCDs."""
    up = lambda n, d: -(-n // d)
    rows = {_abi.FFN_TILE_32: 32, _abi.FFN_TILE_64: 64, _abi.FFN_TILE_128: 128}[tile % DEEP]
    dx = up(T, rows) * up(H, 128)
    dw = 3 * up(H, 128) * up(Hp, 128)
    return 8 * up(dx, 8) + 8 * up(dw, 8)


@pytest.mark.parametrize("size", list(LAST))
def test_tile_of_the_joined_launch(size):
    assert _abi.shared_ffn_last_tile(*size) == LAST[size]


@pytest.mark.parametrize("size", [(1, 5312, 192), (35, 3200, 320), (148, 6464, 64)])
def test_depth_goes_by_both_products(size):
    """Alone each product leaves a CU one workgroup, together they do not."""
    for p in (_abi.FFN_DX, _abi.FFN_WGRAD):
        assert _abi.shared_ffn_tile(*size, p)[0] >= DEEP
    assert _abi.shared_ffn_last_tile(*size) < DEEP and blocks(*size, LAST[size]) > 256


def sizes(n):
    rng = random.Random(11)
    log = lambda top: int(round(math.exp(rng.uniform(0, math.log(top)))))
    for _ in range(n):
        T, H, Hp = log(1 << 17), 64 * log(1024), 64 * log(1024)
        if H * Hp < 1 << 30 and T * max(H, Hp) < 1 << 30:
            yield T, H, Hp


def test_agrees_with_the_products():
    """One launch where neither product is split and their tiles are of a kind."""
    for size in sizes(20000):
        (dx, sx), (dw, sw) = (_abi.shared_ffn_tile(*size, p) for p in (_abi.FFN_DX, _abi.FFN_WGRAD))
        last = _abi.shared_ffn_last_tile(*size)
        small = dx % DEEP <= _abi.FFN_TILE_128
        one = sx == sw == 1 and (small and dw % DEEP == _abi.FFN_TILE_128 or not small and dx == dw)
        assert (last >= 0) == one, size
        if one:
            assert last % DEEP == dx % DEEP, size
            if small:
                assert (last >= DEEP) == (blocks(*size, last) <= 256), size


def test_cases_take_every_form():
    """The sizes that the GPU test runs cover what any size takes, the training microbatch among them."""
    seen = {_abi.shared_ffn_last_tile(*size) for size in sizes(40000)}
    seen.add(_abi.shared_ffn_last_tile(32768, 7168, 2048))
    assert seen - {-1} == set(LAST.values())


def test_cases_take_every_launch_of_the_weight_gradients():
    def alone(*size):
        tile, splits = _abi.shared_ffn_tile(*size, _abi.FFN_WGRAD)
        return (tile, splits > 1) if _abi.shared_ffn_last_tile(*size) < 0 else None

    assert {size: alone(*size) for size in ALONE} == ALONE
    assert {alone(*size) for size in sizes(40000)} - {None} == set(ALONE.values())


def test_sizes_that_there_are_not():
    for bad in ((0, 64, 64), (-1, 64, 64), (4, 96, 64), (4, 64, 0), (1 << 24, 64, 64)):
        assert _abi.shared_ffn_last_tile(*bad) == -1
