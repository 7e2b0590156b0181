"""Host-only checks of shared_ffn and its backward (no GPU needed): what they
refuse before anything is enqueued, and workspace sizes."""
import ctypes
import math
import random

import pytest
import torch

import grouped_gemm_moonep_amd as moonep
from grouped_gemm_moonep_amd import _abi
from shared_ffn_cases import CASES, taken

ARG, CONFIG, SCRATCH, OK = (_abi.MOONEP_ERR_ARG, _abi.MOONEP_ERR_CONFIG, _abi.MOONEP_ERR_SCRATCH,
                            _abi.MOONEP_OK)
A = [0x100000 * i for i in range(1, 16)]        # aligned, never dereferenced on these paths
P3 = ctypes.c_void_p * 3
W = (A[10], A[11], A[12])


def forward(T=4, H=64, Hp=128, x=A[0], w=W, act=0, add=None, y=A[1], ws=A[2], ws_bytes=1 << 30):
    return _abi.lib().moonep_shared_ffn(x, P3(*w), act, add, T, H, Hp, y, ws, ws_bytes, None)


def backward(T=4, H=64, Hp=128, x=A[0], dy=A[1], w=W, act=0, dx=A[2], dw=(A[3], A[4], A[5]),
             dtype=_abi.BF16, ws=A[6], ws_bytes=1 << 30):
    return _abi.lib().moonep_shared_ffn_bwd(x, dy, P3(*w), act, T, H, Hp, dx, P3(*dw), dtype, ws,
                                            ws_bytes, None)


SIZES = [dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=32), dict(H=96), dict(H=65600), dict(Hp=0),
         dict(Hp=100), dict(Hp=65600), dict(H=65536, Hp=16384)]
FORMS = [dict(act=2), dict(act=-1), dict(w=(A[10], None, A[12])), dict(w=(A[10] + 8, A[11], A[12])),
         dict(x=None), dict(x=A[0] + 2), dict(ws=None), dict(ws=A[6] + 16)]


@pytest.mark.parametrize("bad", SIZES)
def test_sizes_refused(bad):
    assert forward(**bad) == CONFIG
    assert backward(**bad) == CONFIG
    n = {**dict(T=4, H=64, Hp=128), **bad}
    assert _abi.lib().moonep_shared_ffn_ws(n["T"], n["H"], n["Hp"]) == -1
    assert _abi.lib().moonep_shared_ffn_bwd_ws(n["T"], n["H"], n["Hp"]) == -1


@pytest.mark.parametrize("bad", FORMS + [dict(y=None), dict(y=A[1] + 8), dict(add=A[3] + 2),
                                         dict(y=A[0]), dict(y=A[11]), dict(y=A[2])])
def test_forward_refuses(bad):
    assert forward(**bad) == ARG


@pytest.mark.parametrize("bad", FORMS + [
    dict(dy=None), dict(dy=A[1] + 4), dict(dx=A[2] + 2), dict(dx=A[0]), dict(dx=A[1]),
    dict(dw=(A[3], None, A[5])), dict(dw=(A[3] + 8, A[4], A[5])), dict(dw=(A[3], A[3], A[5])),
    dict(dw=(A[2], A[4], A[5])), dict(dw=(A[3], A[10], A[5])), dict(dw=(A[3], A[4], A[1])),
    dict(dtype=2)])
def test_backward_refuses(bad):
    assert backward(**bad) == ARG


@pytest.mark.parametrize("bad", [
    dict(y=A[0] + 496), dict(y=A[10] + 64 * 256 - 16), dict(add=A[1] + 16), dict(ws=A[0] - 256),
    dict(ws=A[12] + 256)])
def test_forward_refuses_overlaps(bad):
    assert forward(**bad) == ARG


@pytest.mark.parametrize("bad", [
    dict(dx=A[0] + 16), dict(dx=A[1] - 496), dict(dw=(A[3], A[3] + 64 * 256 - 16, A[5])),
    dict(dw=(A[3], A[3] + 64 * 256, A[5]), dtype=_abi.F32), dict(dw=(A[10] + 16, A[4], A[5])),
    dict(ws=A[1]), dict(ws=A[5] - 256), dict(dw=(A[2] + 496, A[4], A[5]))])
def test_backward_refuses_overlaps(bad):
    assert backward(**bad) == ARG


def test_too_many_tokens_for_the_weight_gradients():
    """The backward addresses the tokens' columns with 31-bit offsets; the forward does not."""
    lib = _abi.lib()
    assert lib.moonep_shared_ffn_bwd_ws((1 << 30) // 7168, 7168, 64) > 0
    assert lib.moonep_shared_ffn_bwd_ws((1 << 30) // 7168 + 1, 7168, 64) == -1
    assert lib.moonep_shared_ffn_ws((1 << 30) // 7168 + 1, 7168, 64) > 0


def test_workspace_sizes_and_scratch():
    lib = _abi.lib()
    for T, H, Hp in [(1, 64, 64), (8, 7168, 2048), (1024, 7168, 2048), (8168, 1024, 2048),
                     (32768, 7168, 2048), (33, 65536, 64)]:
        f, b = lib.moonep_shared_ffn_ws(T, H, Hp), lib.moonep_shared_ffn_bwd_ws(T, H, Hp)
        assert f >= 2 * T * Hp and b >= 6 * T * Hp
        assert forward(T=T, H=H, Hp=Hp, ws_bytes=f - 1) == SCRATCH
        assert backward(T=T, H=H, Hp=Hp, ws_bytes=b - 1) == SCRATCH
    assert lib.moonep_shared_ffn_ws(0, 64, 64) == lib.moonep_shared_ffn_bwd_ws(0, 64, 64) == 0
    assert forward(T=0, x=None, y=None, ws=None) == OK


def test_binding_refuses():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = [torch.zeros((64, 128), dtype=torch.bfloat16) for _ in range(3)]
    for f in (lambda: moonep.shared_ffn(x, w),                           # on the host
              lambda: moonep.shared_ffn(x, w, act="relu"),
              lambda: moonep.shared_ffn(x, w[:2]),
              lambda: moonep.shared_ffn_bwd(x, x, [t[None] for t in w])):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(moonep.MoonepError):
        moonep.shared_ffn_workspace(4, 96, 64, device="cpu")
    with pytest.raises(moonep.MoonepError):
        moonep.shared_ffn_bwd_workspace(1 << 20, 7168, 64, device="cpu")


def test_cases_take_every_tile():
    """The sizes that the GPU test runs cover what any size takes."""
    covered = set().union(*(taken(*c) for c in CASES))
    rng = random.Random(7)
    size = lambda top: 64 * int(round(math.exp(rng.uniform(0, math.log(top)))))
    for _ in range(40000):
        H, Hp = size(1024), size(1024)
        T = int(round(math.exp(rng.uniform(0, math.log(1 << 17)))))
        if H * Hp < 1 << 30:
            assert taken(T, H, Hp) <= covered, (T, H, Hp)


def test_tile_query_refuses():
    lib, n = _abi.lib(), ctypes.c_int32()
    f = lib.moonep_shared_ffn_tile
    assert f(4, 64, 64, 0, ctypes.byref(n)) >= 0 and n.value == 1
    for bad in ((0, 64, 64, 0), (4, 96, 64, 0), (4, 64, 0, 1), (4, 64, 64, 5), (4, 64, 64, -1),
                (1 << 24, 64, 64, 2)):
        assert f(*bad, ctypes.byref(n)) == -1
    assert f(1 << 24, 64, 64, 0, ctypes.byref(n)) >= 0      # the forward takes more tokens
    assert f(4, 64, 64, 0, None) == -1
