"""shared_ffn and shared_ffn_bwd against the oracle in the norm of the error
(bounds and reasons: shared_ffn_norms), at sizes whose sums are long or cut into
splits."""
import numpy as np
import pytest
import torch

from gpu_util import log
from grouped_gemm_moonep_amd import shared_ffn, shared_ffn_bwd
from shared_ffn_norms import results
from test_gpu_shared_ffn import draw, wide

pytestmark = pytest.mark.gpu

SIZES = [
    (257, 64, 1024), (100, 1024, 2048), (40, 7168, 512), (300, 1984, 704), (900, 128, 192),
    (802, 64, 3648), (148, 6464, 64), (35, 11584, 832), (269, 11328, 64),   # small tiles, splits of K
    (12301, 128, 192), (6000, 1088, 512), (33013, 576, 64),                 # the tokens in splits
    (1100, 2048, 1024), (8168, 1024, 2048), (4200, 1024, 2112),             # large tiles
    (132, 25088, 64), (407, 16448, 320), (778, 9408, 320),                  # dX beside them
]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,H,Hp", SIZES)
def test_norm_of_the_error(T, H, Hp, f32):
    act = "gelu_tanh" if T % 2 else "silu"
    x, w, _, dy = draw(T, H, Hp, seed=T)
    log(f"norms T={T} H={H} Hp={Hp} {act} f32={f32}")
    dw = tuple(torch.full((H, Hp), 0.5, device="cuda") for _ in range(3)) if f32 else None
    got = dict(zip(("dWg", "dWu", "dWd"), shared_ffn_bwd(x, dy, w, act=act, dw=dw)[1]))
    if not f32:
        got["y"], got["dx"] = shared_ffn(x, w, act=act), shared_ffn_bwd(x, dy, w, act=act)[0]
    want = results(wide(x), wide(dy), [wide(t) for t in w], act, f32)
    of = {n: float(np.linalg.norm(wide(t) - want[n][0])) / want[n][1] for n, t in got.items()}
    log("of the bound: " + ", ".join(f"{n} {r:.3f}" for n, r in of.items()))
    assert max(of.values()) <= 1.0, of
