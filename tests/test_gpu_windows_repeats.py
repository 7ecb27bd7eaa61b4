"""Calls whose work is cut between CTAs give the same bits whichever of them ends last: units of one and of two tiles of
rows in two to four parts (joined by the last CTA with its own part still in its accumulators) and in many (joined from
the workspace), and key tiles of the gradient in pieces.  Each call is repeated beside other work, which changes the order
in which CTAs begin and end, and replayed from a graph."""
import pytest
import torch

import audio_video_flow_gb300 as h3
from test_gpu_windows import Paged, draw, ok, starts, window_case, ws_of

pytestmark = pytest.mark.gpu


def document(S, H, Hk, w):
    q, k, v = window_case(S, H, Hk, S + H)
    o, lse = torch.empty(S, H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, S, device="cuda")
    ws = ws_of(h3.h3_attention_window_workspace_bytes(S, H, Hk))
    return lambda: h3.h3_attention_window(h3.make_window(**w), S, H, Hk, q, q.stride(0), 128, k, v, k.stride(0), 128, o,
                                          lse, ws), [o, lse]


def cached(lengths, new, H, Hk, page, w):
    c = Paged(lengths, Hk, page, sum(lengths))
    rows = sum(new)
    q = draw(rows, H, torch.Generator().manual_seed(5))
    start = starts(new)
    o, lse = torch.empty(rows, H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, rows, device="cuda")
    ws = ws_of(h3.h3_attention_cached_workspace_bytes(c.cache, rows, H))
    return lambda: h3.h3_attention_cached(c.cache, h3.make_window(**w), rows, H, start, q, q.stride(0), 128, o, lse,
                                          ws), [o, lse]


def gradient(S, H, Hk, w):
    q, k, v = window_case(S, H, Hk, S + H)
    o, lse = torch.empty(S, H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, S, device="cuda")
    ws = ws_of(h3.h3_attention_window_workspace_bytes(S, H, Hk))
    window = h3.make_window(**w)
    h3.h3_attention_window(window, S, H, Hk, q, q.stride(0), 128, k, v, k.stride(0), 128, o, lse, ws)
    d_o = draw(S, H, torch.Generator().manual_seed(6)).contiguous()
    grads = [torch.empty_like(t) for t in (q, k, v)]
    back = ws_of(h3.h3_attention_window_backward_workspace_bytes(S, H, Hk))
    ok()
    return lambda: h3.h3_attention_window_backward(window, S, H, Hk, q, q.stride(0), 128, k, v, k.stride(0), 128, o, d_o,
                                                   lse, grads[0], q.stride(0), 128, grads[1], grads[2], k.stride(0), 128,
                                                   back), grads


def differences(outs, want):
    return sum((a.view(torch.int16) != b.view(torch.int16)).sum() for a, b in zip(outs, want))


def check_repeats(run, outs, info, repeats):
    run()
    ok()
    assert info(h3.h3_last_kernel_info()), h3.h3_last_kernel_info()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    busy = [torch.zeros(64 << 20, device="cuda") for _ in range(2)]    # 256 MB each, more than L2
    small = torch.zeros(1 << 20, device="cuda")
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    for i in range(repeats):
        with torch.cuda.stream(side):
            if i % 3 == 0:
                busy[0].copy_(busy[1])
            for _ in range(i % 5):
                small.add_(1.0)
        for t in outs:
            t.fill_(float("nan"))
        run()
        bad += differences(outs, want)
    ok()
    assert bad.item() == 0, f"{bad.item()} elements differ over {repeats} calls"
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
        run()
    for t in outs:
        t.fill_(float("nan"))
    for _ in range(10):
        with torch.cuda.stream(side):
            busy[0].copy_(busy[1])
        graph.replay()
        bad += differences(outs, want)
    ok()
    assert bad.item() == 0, f"{bad.item()} elements differ in replays"


@pytest.mark.parametrize("make, args", [
    # the last unit of each head has one tile of rows, in two to four parts
    (document, (1100, 8, 8, dict(right=0))),
    (document, (1100, 8, 8, dict())),
    (document, (2100, 8, 8, dict(right=0))),
    (document, (700, 6, 3, dict())),
    (cached, ([8000], [300], 56, 56, 64, dict(right=0))),
    # units of two tiles
    (document, (2500, 57, 57, dict(left=900, right=0, n_first=40))),
    (cached, ([14836], [405], 56, 56, 128, dict(left=12, right=0, n_first=256, unit=405, origin=256))),
    # many parts: chunks, and single rows
    (cached, ([8000], [300], 12, 12, 16, dict(right=0))),
    (cached, ([8000, 3000, 5000], [300, 44, 129], 6, 2, 256, dict(right=0))),
    (cached, ([20000], [1], 4, 2, 64, dict(right=0))),
    (cached, ([5000, 300, 17, 9000], [1, 1, 1, 1], 8, 2, 32, dict(right=0)))])
def test_cut_units_repeat(make, args):
    run, outs = make(*args)
    check_repeats(run, outs, lambda s: s.endswith(" split"), 200)


@pytest.mark.parametrize("S, H, Hk, w", [
    (2600, 2, 1, dict(left=100, right=0, n_first=5)),       # the first key tile alone in pieces
    (2600, 4, 1, dict(right=0)),                            # all of them
    (4099, 24, 4, dict(left=511, right=128, n_first=3))])
def test_gradient_in_pieces_repeats(S, H, Hk, w):
    run, outs = gradient(S, H, Hk, w)
    check_repeats(run, outs, lambda s: not s.endswith("pieces=1,1"), 50)
