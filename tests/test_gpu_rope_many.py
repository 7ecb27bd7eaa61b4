"""Rotary positions where a thread goes round its head loop more than once (a
CTA's heads are more than one batch of loads covers), and where a CTA takes
several rows: each in both types and directions, in place and not, against the
fp64 oracle; and the same calls in the bounds-checked build, together with norm
gradients of many steps.

Run as a script (`python tests/test_gpu_rope_many.py --cases OUT.npz`) it is the
child that runs the bounds-checked cases with whichever library H3_LIBRARY
selects."""
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
for p in (HERE, os.path.dirname(HERE)):
    if p not in sys.path:
        sys.path.insert(0, p)

from test_gpu_train_ops_bounds import _exact  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (torch.bfloat16, 0, 2.0 ** -8), "fp32": (torch.float32, 1, 2.0 ** -24)}
# rows, q heads, k heads, head channels, axes, frequencies
LOOPS = [(1600, 56, 56, 128, 3, 16), (1601, 100, 3, 128, 1, 64), (900, 100, 56, 64, 1, 32)]
FEW = [(5003, 1, 0, 128, 3, 16), (5003, 2, 1, 128, 1, 64), (5003, 1, 0, 26, 1, 13), (5003, 2, 1, 100, 1, 16),
       (9001, 1, 1, 80, 2, 8)]


def info(h3):
    text = h3.h3_last_kernel_info()
    return text, {k: int(v) for k, v in re.findall(r"(\S+)=(\d+)", text)}


def run(h3, shape, dtype, layout, backward, in_place, g):
    S, HQ, HK, width, axes, freqs = shape
    tdtype, code, _ = TYPES[dtype]
    hs = (width + 7) // 8 * 8
    rs = (HQ + HK) * hs
    x = _exact((S, HQ + HK, width), (rs, hs, 1), tdtype, g)
    y = _exact((S, HQ + HK, width), (rs, hs, 1), tdtype, g)
    if in_place:
        y.copy_(x)
    src = y if in_place else x
    pos = torch.randint(-3000, 3000, (S, axes), generator=g, dtype=torch.int32)
    cfg = h3.make_rope_config(width, axes, freqs, layout=layout, dtype=code, magnitude=1.25)
    h3.h3_rope(cfg, S, pos.cuda(), int(backward), src, y, HQ, src[:, HQ:] if HK else None, y[:, HQ:] if HK else None, HK,
               rs, hs, rs, hs)
    return x, y, pos


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("backward, in_place", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("shape", LOOPS + FEW)
def test_long_calls(shape, dtype, layout, backward, in_place):
    import audio_video_flow_gb300 as h3
    from oracle import h3_train_oracle as O
    from test_gpu_train_ops import f64, ok, within
    g = torch.Generator().manual_seed(sum(shape))
    x, y, pos = run(h3, shape, dtype, layout, backward, in_place, g)
    ok()
    text, n = info(h3)
    if shape in FEW:
        assert n["rows/cta"] > 1, text
    else:   # 128 threads of 16-byte pairs, four heads' loads each
        P, V = shape[4] * shape[5], 16 // x.element_size()
        units = (2 * P // V + 1) // 2 + (0 if in_place else -(-(shape[3] - 2 * P) // (2 * V)))
        assert "vectors" in text and n["heads/cta"] > 4 * (128 // units) and n["rows/cta"] == 1, text
    ref, bound = O.rope(f64(x), pos.numpy(), O.rope_frequencies(shape[4], shape[5]), ["half", "interleaved"][layout],
                        magnitude=1.25, backward=backward, half=TYPES[dtype][2])
    within(y, ref, bound, text)


def bounds_cases(h3):
    g = torch.Generator().manual_seed(9)
    out, status = {}, {}

    def done(name, *tensors):
        torch.cuda.synchronize()
        status[name] = h3.h3_sync_check(timeout_ms=60000)
        for i, t in enumerate(tensors):
            out[f"{name}.{i}"] = t.detach().float().cpu().numpy()

    for shape in [(800, 56, 56, 128, 3, 16)] + FEW:
        for dtype in TYPES:
            for layout in (0, 1):
                for in_place in (False, True):
                    y = run(h3, shape, dtype, layout, False, in_place, g)[1]
                    done(f"rope{shape}{dtype}{layout}{in_place}", y)
    for kind in (h3.H3_NORM_RMS, h3.H3_NORM_LAYER):
        for dtype, (tdtype, code, _) in TYPES.items():
            for rows, heads, width in [(9000, 7, 126), (1501, 5, 517), (4703, 1, 2687), (1607, 1, 8190)]:
                hs = (width + 7) // 8 * 8
                st = (heads * hs, hs, 1)
                x, dy, dx = (_exact((rows, heads, width), st, tdtype, g) for _ in range(3))
                gain = torch.randn(width, generator=g).to(tdtype).cuda()
                dg, db = (torch.empty(width, device="cuda") for _ in range(2))
                cfg = h3.make_norm_config(kind, width, code, code)
                ws = torch.empty(h3.h3_norm_backward_workspace_bytes(cfg, rows, heads), dtype=torch.uint8, device="cuda")
                h3.h3_norm_backward(cfg, rows, heads, x, st[0], hs, gain, dy, st[0], hs, dx, st[0], hs, dg, db, ws)
                # (the parameters' gradients are summed over as many CTAs as
                # the build's registers let stay, so they may differ in order)
                done(f"norm{kind}{dtype}{width}", dx)
    return out, status


def test_long_calls_in_the_bounds_checked_build(tmp_path):
    from audio_video_flow_gb300 import _build
    _build.build(bounds=True)
    dst = tmp_path / "bounds.npz"
    r = subprocess.run([sys.executable, os.path.abspath(__file__), "--cases", str(dst)],
                       env=dict(os.environ, H3_LIBRARY="bounds"), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    got = dict(np.load(dst))
    import audio_video_flow_gb300 as h3
    assert os.path.basename(h3.LIB_PATH) == "libh3.so"
    ref, status = bounds_cases(h3)
    assert all(s == 0 for s in status.values()), status
    assert set(got) == set(ref)
    for k, v in ref.items():
        assert np.array_equal(got[k], v, equal_nan=True), f"{k}: bounds-checked build differs"


def _child(dst):
    import audio_video_flow_gb300 as h3
    assert os.path.basename(h3.LIB_PATH) == "libh3_bounds.so"
    out, status = bounds_cases(h3)
    bad = {k: (v, h3.status_string(v)) for k, v in status.items() if v != 0}
    if bad:
        print("bounds-checked build reported:", bad, h3.h3_last_error_site())
        sys.exit(3)
    np.savez(dst, **out)


if __name__ == "__main__":
    if len(sys.argv) == 3 and sys.argv[1] == "--cases":
        _child(sys.argv[2])
