"""Calls without a stream argument run on torch's current stream."""
import types

import pytest
import torch

import audio_video_flow_gb300 as h3


def test_explicit_streams():
    assert h3._stream(12345) == 12345
    assert h3._stream(types.SimpleNamespace(cuda_stream=99)) == 99


def test_before_cuda_is_initialised(monkeypatch):
    """torch.cuda.current_stream(), which initialises CUDA or raises its own error."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    assert h3._stream(None) == 77


@pytest.mark.gpu
def test_current_stream_on_the_gpu():
    torch.zeros(1, device="cuda")
    assert h3._stream(None) == torch.cuda.current_stream().cuda_stream == 0
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert h3._stream(None) == side.cuda_stream != 0
        with torch.cuda.stream(other):
            assert h3._stream(None) == other.cuda_stream
        assert h3._stream(None) == side.cuda_stream
        with torch.cuda.device(torch.cuda.current_device()):
            assert h3._stream(None) == side.cuda_stream
    assert h3._stream(None) == 0
    graph = torch.cuda.CUDAGraph()
    t = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        t.add_(1.0)
        assert h3._stream(None) == side.cuda_stream


@pytest.mark.gpu
def test_a_call_without_a_stream_is_ordered_on_the_current_one():
    """A copy, a call and a copy back on a side stream, without a wait between."""
    n = 1 << 22
    cfg = h3.make_norm_config(h3.H3_NORM_RMS, 1024)
    src = [torch.randn(n // 1024, 1, 1024, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda() for i in (1, 2)]
    want = []
    for t in src:
        y = torch.empty_like(t)
        h3.h3_norm_forward(cfg, n // 1024, 1, t, 1024, 1024, None, None, y, 1024, 1024)
        want.append(y)
    x, y = (torch.empty_like(src[0]) for _ in range(2))
    kept = [torch.empty_like(x) for _ in range(8)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for i, to in enumerate(kept):
            x.copy_(src[i & 1])
            h3.h3_norm_forward(cfg, n // 1024, 1, x, 1024, 1024, None, None, y, 1024, 1024)
            to.copy_(y)
    torch.cuda.synchronize()
    assert h3.h3_sync_check(timeout_ms=60000) == 0
    for i, to in enumerate(kept):
        assert torch.equal(to, want[i & 1])
