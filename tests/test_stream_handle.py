"""The stream that a call without one runs on is torch's current stream."""
import pytest
import torch

from exact_attention_blackwell_tma_gb300 import binding, inputs


@pytest.mark.gpu
@pytest.mark.parametrize("private", [True, False])
def test_calls_run_on_the_current_stream(private, monkeypatch):
    """With torch's raw handle and, where a torch lacks it, with the public one."""
    if not private:
        monkeypatch.setattr(binding, "_raw_stream", None)
    t = {n: x.cuda() for n, x in inputs.small(B=1, H=2, L=300, d=64, seed=191).items()}
    torch.cuda.synchronize()
    ref = binding.forward(t["q"], t["k"], t["v"], causal=True)
    assert binding._stream(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert binding._stream(None) == side.cuda_stream
        got = binding.forward(t["q"], t["k"], t["v"], causal=True)
    assert binding._stream(side) == side.cuda_stream and binding._stream(5) == 5
    torch.cuda.synchronize()
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
