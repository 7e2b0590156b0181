"""Sizes that between them take every tile, ring depth and kind of split of every product of the
shared expert; the host test checks that they do, the GPU test runs them."""
from grouped_gemm_moonep_amd import _abi

CASES = [
    (1, 64, 64), (33, 64, 64), (65, 64, 64), (1, 832, 64), (1, 64, 448), (35, 832, 64), (36, 64, 832),
    (1, 64, 16512), (65, 64, 896), (71, 832, 64), (769, 64, 64), (1, 64, 24896), (33, 64, 11584),
    (1, 832, 5824), (151, 64, 8320), (268, 11328, 64), (33, 34752, 64), (1, 32832, 64),
    (11778, 960, 64), (1, 6720, 4736), (35, 64, 17024), (39, 832, 5824), (1, 11392, 448),
    (35, 11584, 832), (1167, 1152, 832), (33013, 576, 64), (33411, 64, 576), (1, 1600, 36864),
]


def taken(T, H, Hp):
    """{(product, tile, split?)} of a size; ("last", rows) where dX and the weight gradients are
    one launch."""
    got = {}
    for p in _abi.FFN_PRODUCTS:
        tile, splits = _abi.shared_ffn_tile(T, H, Hp, p)
        if tile >= 0:
            got[p] = (tile, splits)
    keys = {(p, t, s > 1) for p, (t, s) in got.items()}
    dx, dw = got.get(_abi.FFN_DX), got.get(_abi.FFN_WGRAD)
    if dx and dw and dx[1] == dw[1] == 1 and dx[0] % 8 <= _abi.FFN_TILE_128 and \
            dw[0] % 8 == _abi.FFN_TILE_128:
        keys.add(("last", dx[0] % 8))
    return keys
