"""What orthogonalize says when it refuses steps, coefficients or eps (no GPU
needed)."""
import pytest

from grouped_gemm_moonep_amd import MUON_COEFFS, _refused_steps


@pytest.mark.parametrize("flat,eps,says", [
    ([MUON_COEFFS] * 7, 1e-7, "7 steps whose a multiply to 5752.9"),
    ([MUON_COEFFS] * 10, 1e-7, "at most 2048"),
    ([], 1e-7, "0 steps, 1 to 16"), ([(1.0, 0.0, 0.0)] * 17, 1e-7, "17 steps, 1 to 16"),
    ([MUON_COEFFS], 0.0, "eps 0.0"), ([MUON_COEFFS], float("nan"), "eps nan"),
    ([(-1.0, 0.0, 0.0)], 1e-7, "not positive"), ([(1.0, float("inf"), 0.0)], 1e-7, "not finite"),
    ([(float("nan"), 0.0, 0.0)], 1e-7, "not finite"),
    ([(2.5, 0.0, 0.0)] * 2, 1e-7, "singular value past 1.99"),
    ([MUON_COEFFS] * 6, 1e-7, None), ([(1.5, -0.5, 0.0)] * 16, 1e-30, None)])
def test_the_reason_names_what_is_refused(flat, eps, says):
    why = _refused_steps(flat, eps)
    assert why is None if says is None else says in why


@pytest.mark.gpu
def test_the_error_carries_the_reason():
    import torch
    from grouped_gemm_moonep_amd import MoonepError, _abi, orthogonalize
    g = torch.ones((4, 6), device="cuda")
    with pytest.raises(MoonepError, match="10 steps whose a multiply to .* at most 2048") as e:
        orthogonalize(g, steps=10)
    assert e.value.status == _abi.MOONEP_ERR_ARG
    with pytest.raises(MoonepError, match="0 steps, 1 to 16"):
        orthogonalize(g, steps=0)
    with pytest.raises(MoonepError, match="^moonep_orthogonalize: [^0-9]*\\(status"):
        orthogonalize(g, ws=torch.empty(1 << 20, dtype=torch.uint8, device="cuda")[1:])
