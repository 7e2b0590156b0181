"""Sizes that between them take every tile and ring depth of the launch that computes dX and the weight
gradients of the shared expert together, and every form of the weight gradients' own launch; the host
test checks that they do, the GPU test runs them."""
from grouped_gemm_moonep_amd import _abi

DEEP = _abi.FFN_TILE_DEEP
# (T, H, H'): tile of dX
LAST = {
    (1, 64, 64): _abi.FFN_TILE_32 + DEEP, (36, 64, 64): _abi.FFN_TILE_64 + DEEP,
    (79, 64, 64): _abi.FFN_TILE_128 + DEEP, (1, 5312, 192): _abi.FFN_TILE_32,
    (35, 3200, 320): _abi.FFN_TILE_64, (148, 6464, 64): _abi.FFN_TILE_128,
    (132, 25088, 64): _abi.FFN_TILE_128X256,
    (407, 16448, 320): _abi.FFN_TILE_256X256,          # last rows of dX: 151 in a whole tile,
    (778, 9408, 320): _abi.FFN_TILE_256X256,           # 10 in a half one
}

# Weight gradients in launches of their own: (tile, in splits?)
ALONE = {
    (3, 64, 448): (_abi.FFN_TILE_128 + DEEP, False), (900, 128, 192): (_abi.FFN_TILE_128 + DEEP, True),
    (2, 64, 11008): (_abi.FFN_TILE_128, False), (802, 64, 3648): (_abi.FFN_TILE_128, True),
    (1100, 2048, 1024): (_abi.FFN_TILE_128X256, False), (6000, 1088, 512): (_abi.FFN_TILE_128X256, True),
    (288, 11136, 64): (_abi.FFN_TILE_256X256, False),
}
