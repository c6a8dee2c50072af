"""The stream that the tensor helpers enqueue on, with torch's raw handle and
without it."""
import pytest
import torch

from tests.parity import say

pytestmark = pytest.mark.gpu


def test_handle_of_the_current_stream(fp8q, monkeypatch):
    say("current stream")
    from fp8_fine_grained_x128_amd import binding
    side = torch.cuda.Stream()
    x = torch.randn((40, 256), device="cuda").to(torch.bfloat16)
    want = fp8q.quantize_act(x)
    for raw in (binding._raw_stream, None):
        monkeypatch.setattr(binding, "_raw_stream", raw)
        assert binding._stream() == torch.cuda.current_stream().cuda_stream
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            assert binding._stream() == side.cuda_stream
            got = fp8q.quantize_act(x)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
