"""Calls of one row: the row stride is never used, so any value will do, as the
head stride with one head."""
import numpy as np
import pytest
import torch

import audio_video_flow_gb300 as h3
from audio_video_flow_gb300 import _build
from test_train_ops_cpu import BACKWARD, FORWARD, ROPE, _call


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return h3.lib()


# Each call has a second fault that is refused after the strides: were the row
# stride looked at, the first status would be the other one.
@pytest.mark.parametrize("stride", [0, 1, 513, -7])
@pytest.mark.parametrize("heads", [1, 4])
def test_row_stride_of_one_row_is_not_looked_at(lib, stride, heads):
    one = dict(n_rows=1, n_heads=heads)
    assert _call(lib.h3_norm_forward, FORWARD, **one, xrs=stride, yrs=stride, y=0x4004) == h3.H3_ERR_ALIGN
    assert _call(lib.h3_norm_backward, BACKWARD, **one, xrs=stride, dyrs=stride, dxrs=stride + 8,
                 ws_bytes=64) == h3.H3_ERR_WORKSPACE
    rope = dict(n_rows=1, q_heads=heads, k_heads=heads, irs=stride, ors=stride + 8)
    assert _call(lib.h3_rope, ROPE, **rope, pos=0x102) == h3.H3_ERR_ALIGN
    assert _call(lib.h3_rope, ROPE, **rope, k_out=0x2000) == h3.H3_ERR_SHAPE
    if heads > 1:   # in place, the head strides still have to agree
        assert _call(lib.h3_norm_forward, FORWARD, **one, xrs=513, yrs=stride, y=0x1000, yhs=136) == h3.H3_ERR_SHAPE
        assert _call(lib.h3_rope, ROPE, **rope, q_out=0x1000, k_out=0x3000, ohs=136) == h3.H3_ERR_SHAPE


@pytest.mark.parametrize("rows", [2, 8])
def test_row_strides_of_more_rows_are(lib, rows):
    for stride, rope_stride, status in ((504, 120, h3.H3_ERR_SHAPE), (513, 129, h3.H3_ERR_ALIGN)):
        changed = dict(n_rows=rows, n_heads=1, cfg=h3.make_norm_config(h3.H3_NORM_LAYER, 512))
        assert _call(lib.h3_norm_forward, FORWARD, **changed, xrs=stride) == status
        assert _call(lib.h3_norm_backward, BACKWARD, **changed, dxrs=stride) == status
        assert _call(lib.h3_rope, ROPE, n_rows=rows, irs=rope_stride) == status


@pytest.mark.gpu
@pytest.mark.parametrize("heads, width", [(1, 1009), (1, 5375), (3, 128), (5, 100)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_one_row_of_any_row_stride(heads, width, dtype):
    """One contiguous row, its stride the tensor's own (no multiple of 16 bytes),
    against the same row under an aligned stride, bit for bit; in place too."""
    tdtype, code = {"bf16": (torch.bfloat16, h3.H3_BF16), "fp32": (torch.float32, h3.H3_FP32)}[dtype]
    hs = width if heads == 1 else (width + 7) // 8 * 8
    g = torch.Generator().manual_seed(width)
    x, dy = (torch.randn(1, heads, hs, generator=g).to(tdtype).cuda() for _ in range(2))
    cfg = h3.make_norm_config(h3.H3_NORM_LAYER, width, code, code)
    rope = h3.make_rope_config(128, 1, 24, dtype=code) if width == 128 else None
    pos = torch.tensor([[77]], dtype=torch.int32, device="cuda")
    ws = torch.empty(h3.h3_norm_backward_workspace_bytes(cfg, 1, heads), dtype=torch.uint8, device="cuda")
    got = []
    for rs in (8192, heads * hs, 3, 0):
        y, dx, z = (torch.full_like(x, 5.0) for _ in range(3))
        dg, db = (torch.full((width,), 9.0, device="cuda") for _ in range(2))
        h3.h3_norm_forward(cfg, 1, heads, x, rs, hs, None, None, y, rs, hs)
        h3.h3_norm_backward(cfg, 1, heads, x, rs, hs, None, dy, rs + 1, hs, dx, rs, hs, dg, db, ws)
        place = x.clone()
        h3.h3_norm_forward(cfg, 1, heads, place, rs, hs, None, None, place, rs + 8, hs)
        assert torch.equal(place[..., :width], y[..., :width])
        if rope is not None:
            h3.h3_rope(rope, 1, pos, 0, x, z, heads, None, None, 0, rs, hs, rs, hs)
        got.append([t.clone() for t in (y, dx, z, dg, db)])
    torch.cuda.synchronize()
    assert h3.h3_sync_check(timeout_ms=60000) == 0
    assert np.isfinite(got[0][0].float().cpu().numpy()).all()
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
