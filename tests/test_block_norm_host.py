"""Host-only checks of block_norm and its backward (no GPU needed): sizes and
arguments refused before anything is enqueued, workspace sizes, and what the
binding refuses."""
import pytest
import torch

import grouped_gemm_moonep_amd as moonep
from grouped_gemm_moonep_amd import _abi

ARG, CONFIG, SCRATCH, OK = (_abi.MOONEP_ERR_ARG, _abi.MOONEP_ERR_CONFIG, _abi.MOONEP_ERR_SCRATCH,
                            _abi.MOONEP_OK)
A = [0x10000 * i for i in range(1, 16)]         # aligned, never dereferenced on these paths


def forward(T=4, W=64, dtype=_abi.F32, h=A[0], y=A[1], y2=None, gate=None, kind=0, w_post=A[2],
            w_pre=A[3], scale=1.0, eps=1e-6, h_out=A[4], u=A[5]):
    return _abi.lib().moonep_block_norm(h, dtype, y, y2, gate, kind, w_post, w_pre, scale, eps, T,
                                        W, h_out, u, None)


def backward(T=4, W=64, dtype=_abi.F32, h=A[0], dh=A[1], du=A[2], y=A[3], y2=None, gate=None,
             kind=0, w_post=A[4], w_pre=A[5], scale=1.0, eps=1e-6, dres=A[6], dy=A[7], dgate=None,
             dw_post=A[8], dw_pre=A[9], ws=A[10], ws_bytes=1 << 30):
    return _abi.lib().moonep_block_norm_bwd(h, dtype, dh, du, y, y2, gate, kind, w_post, w_pre,
                                            scale, eps, T, W, dres, dy, dgate, dw_post, dw_pre, ws,
                                            ws_bytes, None)


NAN = float("nan")
SIZES = [(dict(T=-1), CONFIG), (dict(T=1 << 31), CONFIG), (dict(W=0), CONFIG), (dict(W=12), CONFIG),
         (dict(W=16392), CONFIG), (dict(W=-8), CONFIG)]
FORMS = [(dict(dtype=2), ARG), (dict(kind=4), ARG), (dict(kind=-1), ARG), (dict(kind=1), ARG),
         (dict(gate=A[11]), ARG), (dict(eps=0.0), ARG), (dict(eps=NAN), ARG),
         (dict(eps=float("inf")), ARG), (dict(scale=NAN), ARG), (dict(w_post=A[2] + 4), ARG),
         (dict(w_pre=A[3] + 8), ARG), (dict(y=A[1] + 2), ARG), (dict(y2=A[12] + 8), ARG),
         (dict(kind=1, gate=A[11] + 4), ARG), (dict(kind=3, gate=A[11] + 8), ARG),
         (dict(kind=2, gate=A[11] + 2), ARG)]


@pytest.mark.parametrize("bad,status", SIZES + FORMS + [
    (dict(h=None), ARG), (dict(h=A[0] + 4), ARG), (dict(h_out=None), ARG), (dict(u=None), ARG),
    (dict(w_pre=None), ARG), (dict(y=None), ARG), (dict(y=None, w_post=None), ARG),
    (dict(y=None, w_post=None, w_pre=None, h_out=None, u=None), ARG),
    (dict(y=None, w_post=None, y2=A[12], h_out=None), ARG), (dict(u=A[0]), ARG), (dict(u=A[4]), ARG),
])
def test_forward_refuses(bad, status):
    assert forward(**bad) == status


@pytest.mark.parametrize("bad,status", SIZES + FORMS + [
    (dict(dres=None), ARG), (dict(h=None), ARG), (dict(du=None), ARG), (dict(w_pre=None), ARG),
    (dict(dh=None, du=None, w_pre=None, dw_pre=None), ARG), (dict(dgate=A[12]), ARG),
    (dict(w_post=None), ARG), (dict(y=None, w_post=None, dw_post=None), ARG), (dict(ws=None), ARG),
    (dict(ws=A[10] + 8), ARG), (dict(ws_bytes=100), SCRATCH), (dict(dres=A[7]), ARG),
    (dict(dres=A[2]), ARG), (dict(dres=A[3]), ARG), (dict(dres=A[0]), ARG), (dict(dh=A[1] + 4), ARG),
])
def test_backward_refuses(bad, status):
    assert backward(**bad) == status


@pytest.mark.parametrize("bad", [
    dict(h_out=A[0] + 16), dict(h_out=A[1]), dict(h_out=A[2]), dict(u=A[0] + 512), dict(u=A[1] + 16),
    dict(u=A[3]), dict(u=A[4] + 1008), dict(y2=A[6], h_out=A[6]), dict(kind=1, gate=A[4] + 64),
    dict(kind=3, gate=A[7], u=A[7]), dict(kind=2, gate=A[5] + 4)])
def test_forward_refuses_overlaps(bad):
    assert forward(**bad) == ARG


@pytest.mark.parametrize("bad", [
    dict(dres=A[1] + 16), dict(dres=A[2] + 496), dict(dy=A[6] + 1008), dict(dy=A[0]),
    dict(dy=A[3] + 16), dict(dw_post=A[9]), dict(dw_pre=A[5]), dict(ws=A[0] + 256), dict(dw_post=A[10]),
    dict(kind=1, gate=A[11], dgate=A[11]), dict(kind=2, gate=A[11], dgate=A[7] + 500),
    dict(y2=A[12], dres=A[12] + 256)])
def test_backward_refuses_overlaps(bad):
    assert backward(**bad) == ARG


def test_no_rows_need_no_pointers():
    assert forward(T=0, h=None, h_out=None, u=None) == OK


def test_workspace_sizes():
    ws = _abi.lib().moonep_block_norm_bwd_ws
    assert ws(-1, 64) == ws(4, 12) == ws(1 << 31, 64) == ws(4, 16392) == -1
    assert ws(0, 64) == 0
    for W in (8, 1024, 1032, 7168, 16384):
        got = [ws(T, W) for T in (1, 2, 64, 4096, 32768, (1 << 31) - 1)]
        assert all(b > 0 and b % (12 * W) == 0 for b in got) and got == sorted(got)
        # bounded by the launch, whatever the number of rows
        assert got[-1] <= 12 * W * 2048


def test_binding_refuses():
    h = torch.zeros((4, 64))
    y = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.ones(64)
    for bad in (dict(h=h, y=y, w_post=w),                      # on the host
                dict(h=h)):
        with pytest.raises(ValueError):
            moonep.block_norm(**bad)
    with pytest.raises(moonep.MoonepError):
        moonep.block_norm_bwd_workspace(4, 12, device="cpu")
