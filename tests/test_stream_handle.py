"""The handle of torch's current stream that every call passes on."""
import types

import pytest


def test_without_torchs_raw_getter_the_documented_one_serves(monkeypatch):
    import torch
    import moe_glue_amd as mg

    monkeypatch.setattr(mg, "_raw_stream", None)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: types.SimpleNamespace(cuda_stream=1000 + index))
    assert mg._stream(torch.device("cuda", 3)) == 1003
    assert mg._stream(torch.device("cuda", 0)) == 1000


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [True, False])
def test_the_handle_is_the_current_streams(monkeypatch, raw):
    import torch
    import moe_glue_amd as mg

    monkeypatch.setattr(mg, "_raw_stream", None)
    if not raw:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    dev = torch.device("cuda", 0)
    x = torch.randn(64, 64, device=dev).bfloat16()
    w = torch.ones(64, device=dev).bfloat16()
    assert mg._stream(dev) == torch.cuda.default_stream(dev).cuda_stream
    side = torch.cuda.Stream(device=dev)
    with torch.cuda.stream(side):
        assert mg._stream(dev) == side.cuda_stream
        a = mg.rmsnorm(x, w)[0]
    assert mg._stream(dev) == torch.cuda.default_stream(dev).cuda_stream
    b = mg.rmsnorm(x, w)[0]
    torch.cuda.synchronize()
    assert torch.equal(a, b)
