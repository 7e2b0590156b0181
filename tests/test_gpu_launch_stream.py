"""The stream and device that the training-step calls launch on, by torch's
public functions too."""
import pytest
import torch

import grouped_gemm_moonep_amd as moonep

pytestmark = pytest.mark.gpu


def test_public_functions_name_the_same_stream_and_device():
    i = torch.cuda.current_device()
    assert moonep._current_device() == i
    for stream in (torch.cuda.default_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            assert moonep._raw_stream(i) == moonep._stream_of(i) == stream.cuda_stream


def test_calls_without_the_private_functions(monkeypatch):
    buf = moonep.Buffer(R=1, S=5, K=2, E=8, H=64, Hp=64)
    x = torch.randn((1, 5, 8), device="cuda")
    want = buf.route(x)
    monkeypatch.setattr(moonep, "_raw_stream", moonep._stream_of)
    monkeypatch.setattr(moonep, "_current_device", torch.cuda.current_device)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = buf.route(x)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    buf.destroy()
