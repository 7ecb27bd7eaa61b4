"""The window and cache operators in the bounds-checked build (libh3_bounds.so): every checked global access lies in the
buffer that the call's arguments describe, and the results equal the normal build's bit for bit.

Run as a script (`python tests/test_gpu_windows_bounds.py --cases OUT.npz`) it is the child that runs the cases with
whichever library H3_LIBRARY selects.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
for path in (ROOT, HERE):
    if path not in sys.path:
        sys.path.insert(0, path)

pytestmark = pytest.mark.gpu


def run_cases(h3):
    import test_gpu_windows as T
    out, status = {}, {}

    def done(name, *tensors):
        torch.cuda.synchronize()
        status[name] = h3.h3_sync_check(timeout_ms=60000)
        for i, t in enumerate(tensors):
            out[f"{name}.{i}"] = t.detach().float().nan_to_num(-77.0).cpu().numpy()

    g = torch.Generator().manual_seed(1)
    for S, H, Hk, w in [(1, 1, 1, {}), (300, 6, 2, dict(left=70, right=0, n_first=3)), (2600, 2, 1, dict(left=100, right=0, n_first=5)),
                        (601, 3, 3, dict(left=1, right=1, unit=33, origin=10, n_first=140))]:
        q, k, v = T.window_case(S, H, Hk, S, gap=8)
        o, lse = T.run_window(w, q, k, v)
        d_o = torch.randn(S, H, 128, generator=g).to(torch.bfloat16).cuda()
        done(f"window{S}", o, lse, *T.run_backward(w, q, k, v, o, lse, d_o, gap=8))
    for lengths, new, H, Hk, page, w in T.CACHED:
        c = T.Paged(lengths, Hk, page, 5)
        q, k, v = T.draw(sum(new) + 2, H, g), T.draw(sum(new) + 2, Hk, g), T.draw(sum(new) + 2, Hk, g)
        start = T.starts(new)
        h3.h3_cache_append(c.cache, q.shape[0], start, k, v, k.stride(0), k.stride(1), c.w)
        o, lse = T.run_cached(c, w, q, start, H)
        h3.h3_cache_weights(c.cache, h3.make_window(**w), q.shape[0], H, start, q, q.stride(0), q.stride(1), lse, c.w, c.w)
        budget = max(1, max(lengths) // 2)
        to = T.Paged([min(n, budget) for n in lengths], Hk, 16, 6)
        kept = torch.empty(len(lengths), Hk, budget, dtype=torch.int32, device="cuda")
        h3.h3_cache_evict(c.cache, to.cache, budget, budget // 4, budget // 2, c.w, to.w, kept, to.length)
        done(f"cached{len(out)}", o, lse, c.k, c.w, kept, to.length, to.k, to.v, to.w)
    return out, status


def test_accesses_stay_in_bounds_and_change_nothing(tmp_path):
    import audio_video_flow_gb300 as h3
    from audio_video_flow_gb300 import _build
    _build.build(bounds=True)
    path = str(tmp_path / "bounds.npz")
    env = dict(os.environ, H3_LIBRARY="bounds")
    r = subprocess.run([sys.executable, os.path.abspath(__file__), "--cases", path], env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    want, status = run_cases(h3)
    assert all(s == 0 for s in status.values()), status
    got = np.load(path)
    assert set(got.files) == set(want)
    for name in want:
        assert np.array_equal(got[name], want[name]), name


if __name__ == "__main__":
    import audio_video_flow_gb300 as h3
    assert os.path.basename(h3.LIB_PATH) == "libh3_bounds.so"
    cases, status = run_cases(h3)
    bad = {k: v for k, v in status.items() if v}
    if bad:
        print(bad, h3.h3_last_error_site())
        sys.exit(1)
    np.savez(sys.argv[sys.argv.index("--cases") + 1], **cases)
