"""Sizes that do not fit the C calls' 32-bit arguments are refused, not cut to their low bits."""
import pytest

import grouped_gemm_moonep_amd as moonep


@pytest.mark.parametrize("big", [1 << 31, (1 << 32) + 64, 1 << 40])
def test_sizes_past_32_bits(big):
    for call, sizes in ((moonep.shared_ffn_workspace, (1, big, 64)),
                        (moonep.shared_ffn_workspace, (1, 64, big)),
                        (moonep.shared_ffn_bwd_workspace, (1, big, 64)),
                        (moonep.shared_ffn_bwd_workspace, (1, 64, big)),
                        (moonep.block_norm_bwd_workspace, (1, big))):
        with pytest.raises(moonep.MoonepError):
            call(*sizes, device="cpu")
