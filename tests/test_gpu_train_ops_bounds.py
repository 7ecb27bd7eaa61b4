"""The training-side operators in the bounds-checked build (libh3_bounds.so):
every checked global access must lie in the buffer that the call's arguments
describe, and the results must equal the normal build's bit for bit.  The
shapes end inside tiles, chunks and vectors, with gaps between rows.

Run as a script (`python tests/test_gpu_train_ops_bounds.py --cases OUT.npz`)
it is the child that runs the cases with whichever library H3_LIBRARY selects.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

pytestmark = pytest.mark.gpu


def _exact(shape, strides, dtype, g):
    """A strided view whose storage ends with its last element."""
    size = 1 + sum((n - 1) * s for n, s in zip(shape, strides))
    flat = torch.randn(size, generator=g).to(dtype).cuda()
    return flat.as_strided(shape, strides)


def run_cases(h3):
    g = torch.Generator().manual_seed(5)
    out, status = {}, {}

    def done(name, *tensors):
        torch.cuda.synchronize()
        status[name] = h3.h3_sync_check(timeout_ms=60000)
        for i, t in enumerate(tensors):
            out[f"{name}.{i}"] = t.detach().float().cpu().numpy()

    bf, f32 = torch.bfloat16, torch.float32
    for S, H, gap in [(1, 1, 0), (129, 3, 8), (300, 2, 0)]:
        rs, hs = H * (128 + gap), 128 + gap
        q, k, v = (_exact((S, H, 128), (rs, hs, 1), bf, g) for _ in range(3))
        o, d_o = (_exact((S, H, 128), (H * 128, 128, 1), bf, g) for _ in range(2))
        lse = torch.empty(H, S, device="cuda")
        h3.h3_attention(S, H, q, k, v, rs, hs, o, lse)
        dq, dk, dv = (_exact((S, H, 128), (rs, hs, 1), bf, g) for _ in range(3))
        ws = torch.empty(h3.h3_attention_backward_workspace_bytes(S, H), dtype=torch.uint8, device="cuda")
        h3.h3_attention_backward(S, H, q, k, v, rs, hs, o, d_o, lse, dq, dk, dv, rs, hs, ws)
        done(f"attention{S}x{H}", dq, dk, dv)
    for dtype, code in [(bf, h3.H3_BF16), (f32, h3.H3_FP32)]:
        for layout in (h3.H3_ROPE_HALF, h3.H3_ROPE_INTERLEAVED):
            for width, axes, freqs in [(128, 3, 16), (26, 1, 13), (100, 1, 16), (80, 2, 8)]:
                S, HQ, HK = 13, 3, 2
                hs = (width + 7) // 8 * 8
                x = _exact((S, HQ + HK, width), ((HQ + HK) * hs, hs, 1), dtype, g)
                y = _exact((S, HQ + HK, width), ((HQ + HK) * hs, hs, 1), dtype, g)
                pos = torch.randint(0, 1000, (S, axes), generator=g, dtype=torch.int32).cuda()
                cfg = h3.make_rope_config(width, axes, freqs, layout=layout, dtype=code)
                h3.h3_rope(cfg, S, pos, 0, x, y, HQ, x[:, HQ:], y[:, HQ:], HK, x.stride(0), hs, y.stride(0), hs)
                done(f"rope{code}{layout}{width}", y)
        for kind in (h3.H3_NORM_RMS, h3.H3_NORM_LAYER):
            for rows, heads, width in [(1, 1, 1), (37, 1, 130), (9, 4, 128), (21, 1, 1009), (11, 1, 2300), (5, 1, 5376),
                                       (7, 1, 8190)]:
                hs = (width + 7) // 8 * 8
                st = (heads * hs, hs, 1)
                x, dy, y, dx = (_exact((rows, heads, width), st, dtype, g) for _ in range(4))
                gain, bias = (torch.randn(width, generator=g).to(dtype).cuda() for _ in range(2))
                dg, db = (torch.empty(width, device="cuda") for _ in range(2))
                cfg = h3.make_norm_config(kind, width, code, code)
                ws = torch.empty(h3.h3_norm_backward_workspace_bytes(cfg, rows, heads), dtype=torch.uint8, device="cuda")
                h3.h3_norm_forward(cfg, rows, heads, x, st[0], hs, gain, bias, y, st[0], hs)
                h3.h3_norm_backward(cfg, rows, heads, x, st[0], hs, gain, dy, st[0], hs, dx, st[0], hs, dg, db, ws)
                done(f"norm{code}{kind}{width}", y, dx, dg, db)
    return out, status


def test_bounds_checked_build_matches_and_reports_nothing(tmp_path):
    assert torch.cuda.is_available()
    from audio_video_flow_gb300 import _build
    _build.build(bounds=True)
    dst = tmp_path / "bounds.npz"
    r = subprocess.run([sys.executable, os.path.abspath(__file__), "--cases", str(dst)],
                       env=dict(os.environ, H3_LIBRARY="bounds"), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    got = dict(np.load(dst))
    import audio_video_flow_gb300 as h3
    assert os.path.basename(h3.LIB_PATH) == "libh3.so"
    ref, status = run_cases(h3)
    assert all(s == 0 for s in status.values()), status
    assert set(got) == set(ref)
    for k, v in ref.items():
        assert np.array_equal(got[k], v, equal_nan=True), f"{k}: bounds-checked build differs"


def _child(dst):
    import audio_video_flow_gb300 as h3
    assert os.path.basename(h3.LIB_PATH) == "libh3_bounds.so"
    out, status = run_cases(h3)
    bad = {k: (v, h3.status_string(v)) for k, v in status.items() if v != 0}
    if bad:
        print("bounds-checked build reported:", bad, h3.h3_last_error_site())
        sys.exit(3)
    np.savez(dst, **out)


if __name__ == "__main__":
    if len(sys.argv) == 3 and sys.argv[1] == "--cases":
        _child(sys.argv[2])
