"""Host-only checks of the training-step entry points (no GPU needed): what
they refuse before anything is enqueued, workspace sizes, and the combine
gradient's grid under a CU budget."""
import ctypes

import pytest
import torch

import moonep_synth as synth
from grouped_gemm_moonep_amd import (MUON_COEFFS, MoonepError, _abi, orthogonalize,
                                     orthogonalize_workspace)

ARG, CONFIG, SCRATCH = _abi.MOONEP_ERR_ARG, _abi.MOONEP_ERR_CONFIG, _abi.MOONEP_ERR_SCRATCH
FAKE = 0x10000                    # aligned, never dereferenced on these paths


def test_handle_is_required():
    lib = _abi.lib()
    plan = _abi.MoonepPlan(*([FAKE] * len(_abi.PLAN_ARRAYS)))
    assert lib.moonep_route(None, FAKE, _abi.F32, None, 0, 1, 1.0, FAKE, FAKE, None) == ARG
    assert lib.moonep_route_bwd(None, FAKE, _abi.F32, 0, 1, 1.0, FAKE, FAKE, FAKE, None) == ARG
    assert lib.moonep_combine_bwd(None, ctypes.byref(plan), FAKE, 8, FAKE, FAKE, FAKE, FAKE,
                                  None) == ARG


def ortho(n=1, rows=8, cols=8, g=FAKE, dtype=_abi.F32, coeffs=MUON_COEFFS * 5, steps=5, eps=1e-7,
          out=FAKE, ws=FAKE, ws_bytes=None):
    c = None if coeffs is None else (ctypes.c_float * len(coeffs))(*coeffs)
    if ws_bytes is None:
        ws_bytes = max(_abi.lib().moonep_orthogonalize_ws(n, rows, cols), 0)
    return _abi.lib().moonep_orthogonalize(g, dtype, n, rows, cols, c, steps, eps, out, ws, ws_bytes,
                                           None)


@pytest.mark.parametrize("bad,status", [
    (dict(n=-1), CONFIG), (dict(rows=0), CONFIG), (dict(cols=0), CONFIG),
    (dict(rows=65537), CONFIG), (dict(rows=65536, cols=8192), CONFIG),
    (dict(dtype=2), ARG), (dict(coeffs=None), ARG), (dict(steps=0), ARG),
    (dict(steps=17, coeffs=(1.0, 0.0, 0.0) * 17), ARG),
    (dict(eps=0.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(coeffs=(0.0, 1.0, 1.0) * 5), ARG), (dict(coeffs=(float("nan"), 1.0, 1.0) * 5), ARG),
    (dict(coeffs=(1.0, float("nan"), 0.0) * 5), ARG), (dict(coeffs=(1.0, 0.0, float("inf")) * 5), ARG),
    (dict(steps=1, coeffs=(0.1, 1.0, 0.0)), ARG),          # 1 + b / a = 11
    (dict(steps=2, coeffs=(2.5, 0.0, 0.0) * 2), ARG),      # singular values up to 2.5 after one
    (dict(steps=1, coeffs=(1.0, -20.0, 20.0)), ARG),       # 1 - 20 l + 20 l^2 is -4 at l = 1/2
    (dict(steps=3, coeffs=(0.5, 0.4, 0.0) * 3), ARG),      # R at most 1.8, their product 5.8
    (dict(steps=7, coeffs=MUON_COEFFS * 7), ARG),          # 3.4445^7 > 2048
    (dict(g=None), ARG), (dict(out=None), ARG), (dict(ws=None), ARG), (dict(g=FAKE + 2), ARG),
    (dict(out=FAKE + 1), ARG), (dict(ws=FAKE + 16), ARG), (dict(ws_bytes=100), SCRATCH),
])
def test_orthogonalize_refuses(bad, status):
    assert ortho(**bad) == status


@pytest.mark.parametrize("coeffs", [MUON_COEFFS * 6, (1.5, -0.5, 0.0) * 16, (1.0, 0.0, 0.0) * 16,
                                    (2.5, 0.0, 0.0), (1.875, -1.25, 0.375) * 10,
                                    (8.0, -22.0, 15.8) + (3.9, -2.8, 0.5) * 2])
def test_orthogonalize_takes_converging_coefficients(coeffs):
    assert ortho(n=0, steps=len(coeffs) // 3, coeffs=coeffs) == _abi.MOONEP_OK


def test_orthogonalize_of_nothing_is_nothing():
    assert ortho(n=0, g=None, out=None, ws=None, ws_bytes=0) == _abi.MOONEP_OK


def test_orthogonalize_workspace_sizes():
    ws = _abi.lib().moonep_orthogonalize_ws
    assert ws(0, 8, 8) == 0
    # one matrix: X_0 twice and five m x m matrices, each value a pair of 16 bits in blocks of 32
    assert ws(1, 64, 128) == 2048 + 4 * (64 * 128 + 128 * 64 + 5 * 64 * 64)
    assert ws(1, 128, 64) == ws(1, 64, 128)
    # at most about eight rounds of tiles are taken at a time
    assert ws(1 << 20, 64, 128) == 2048 * ws(1, 64, 128)
    assert ws(1, 7168, 2048) < 4 * (2 * 7168 * 2048 + 5 * 2048 * 2048) + 8192
    for bad in ((-1, 8, 8), (1, 0, 8), (1, 8, 65537), (1, 65536, 8192)):
        assert ws(*bad) == -1


def test_orthogonalize_binding_refuses():
    g = torch.zeros(4, 4)
    with pytest.raises(ValueError, match="device tensor"):
        orthogonalize(g)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        orthogonalize(g.half())
    with pytest.raises(ValueError, match="rows"):
        orthogonalize(torch.zeros(4))
    with pytest.raises(ValueError, match="coeffs"):
        orthogonalize(g, coeffs=[(1.0, 2.0, 3.0)] * 4)
    with pytest.raises(ValueError, match="coeffs"):
        orthogonalize(g, coeffs=[])
    with pytest.raises(MoonepError) as e:
        orthogonalize_workspace(1, 0, 4, device="cpu")
    assert e.value.status == CONFIG


@pytest.mark.parametrize("name", sorted(synth.WORKLOADS))
def test_cu_budget_caps_the_combine_gradient(name):
    w = synth.WORKLOADS[name]
    cfg = lambda n=0: _abi.config(w.R, w.S, w.K, w.E, w.B, w.H, w.Hp, w.token_padding, n)
    for W in (8, 72, 136, 264, w.H):
        free = _abi.launch_grid(cfg(), _abi.GRID_COMBINE_BWD, W)
        lanes = next(g for g in (8, 16, 32, 64) if g >= W // 8 or g == 64)
        assert free * 256 >= w.R * w.S * w.K * lanes       # every (token, k) has its lanes
        for n in (1, 3, 32):
            assert 1 <= _abi.launch_grid(cfg(n), _abi.GRID_COMBINE_BWD, W) <= min(free, 8 * n)
    for W in (0, -8, 12):
        assert _abi.launch_grid(cfg(), _abi.GRID_COMBINE_BWD, W) == -1
