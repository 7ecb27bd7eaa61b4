"""Forms of the window and cache calls that a program meets: head-major tensors, no log-sum-exp asked for, no new rows at
all, the most sequences, and captured calls that follow the table, the lengths and the rows of a replay."""
import numpy as np
import pytest
import torch

import audio_video_flow_gb300 as h3
from oracle import h3_window_oracle as O
from test_gpu_windows import (Paged, backward_inputs, check_backward, check_cached, check_window, draw, f64, ok, run_cached,
                              run_window, starts, window_case, within, ws_of)

pytestmark = pytest.mark.gpu

CASES = [(200, 4, 2, dict(left=50, right=0, n_first=3)), (700, 6, 3, dict(right=0)), (1, 3, 1, dict())]


def head_major(t):
    return t.transpose(0, 1).contiguous().transpose(0, 1)


@pytest.mark.parametrize("S, H, Hk, w", CASES)
def test_head_major(S, H, Hk, w):
    q, k, v = window_case(S, H, Hk, S)
    o, lse = run_window(w, q, k, v)
    qt, kt, vt = (head_major(t) for t in (q, k, v))
    o2, lse2 = run_window(w, qt, kt, vt)
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_window(w, q, k, v, o, lse, f"S={S}")
    o, lse, d_o = backward_inputs(w, q, k, v, torch.Generator().manual_seed(S))
    grads = [head_major(torch.full_like(t, 7.0)) for t in (q, k, v)]
    dq, dk, dv = grads
    h3.h3_attention_window_backward(h3.make_window(**w), S, H, Hk, qt, qt.stride(0), qt.stride(1), kt, vt, kt.stride(0),
                                    kt.stride(1), o, d_o, lse, dq, dq.stride(0), dq.stride(1), dk, dv, dk.stride(0),
                                    dk.stride(1), ws_of(h3.h3_attention_window_backward_workspace_bytes(S, H, Hk)))
    ok()
    check_backward(w, q, k, v, o, lse, d_o, grads, f"S={S}")


def test_head_major_rows_of_a_cache():
    lengths, new, H, Hk = [300, 90, 41], [100, 1, 41], 4, 2
    c = Paged(lengths, Hk, 32, 5)
    g = torch.Generator().manual_seed(6)
    q, k, v = draw(sum(new), H, g), draw(sum(new), Hk, g), draw(sum(new), Hk, g)
    start = starts(new)
    for s, n in enumerate(new):
        at = sum(new[:s])
        c.data[s] = (torch.cat([c.data[s][0][:-n], k[at:at + n]]), torch.cat([c.data[s][1][:-n], v[at:at + n]]), None)
    kt, vt, qt = head_major(k), head_major(v), head_major(q)
    h3.h3_cache_append(c.cache, sum(new), start, kt, vt, kt.stride(0), kt.stride(1), c.w)
    o, lse = run_cached(c, dict(right=0), qt, start, H)
    weights = []
    for t in (q, qt):
        weights.append(c.w.clone())
        h3.h3_cache_weights(c.cache, h3.make_window(right=0), sum(new), H, start, t, t.stride(0), t.stride(1), lse,
                            weights[-1], weights[-1])
    ok()
    check_cached(c, dict(right=0), q, new, H, o, lse, "head-major")
    assert torch.equal(weights[0], weights[1])


@pytest.mark.parametrize("S, H, Hk, w", CASES)
def test_without_log_sum_exp(S, H, Hk, w):
    q, k, v = window_case(S, H, Hk, S)
    want, _ = run_window(w, q, k, v)
    o = torch.full((S, H * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    h3.h3_attention_window(h3.make_window(**w), S, H, Hk, q, q.stride(0), 128, k, v, k.stride(0), 128, o, None,
                           ws_of(h3.h3_attention_window_workspace_bytes(S, H, Hk)))
    ok()
    assert torch.equal(o.view_as(want), want)
    c = Paged([3000, S], Hk, 16, 4)
    new = [min(2, S), S]
    q = draw(sum(new), H, torch.Generator().manual_seed(1))
    want, _ = run_cached(c, w, q, starts(new), H)
    o = torch.full((sum(new), H * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    h3.h3_attention_cached(c.cache, h3.make_window(**w), sum(new), H, starts(new), q, q.stride(0), 128, o, None,
                           ws_of(h3.h3_attention_cached_workspace_bytes(c.cache, sum(new), H)))
    ok()
    assert torch.equal(o.view_as(want), want)


@pytest.mark.parametrize("rows", [1, 700])
def test_no_sequence_has_new_rows(rows):
    """A padded batch whose rows all lie behind the last sequence."""
    lengths = [400, 0, 33]
    c = Paged(lengths, 2, 16, 4)
    q = draw(rows, 4, torch.Generator().manual_seed(1))
    start = torch.zeros(4, dtype=torch.int32, device="cuda")
    before = [t.clone() for t in (c.k, c.v, c.w)]
    h3.h3_cache_append(c.cache, rows, start, q[:, :2], q[:, 2:], q.stride(0), 128, c.w)
    o, lse = run_cached(c, dict(right=0), q, start, 4)
    assert (o == 7.0).all() and (lse == 7.0).all()
    out = torch.full_like(c.w, 5.0)
    for w_in, w_out in ((c.w, out), (c.w, c.w)):
        h3.h3_cache_weights(c.cache, h3.make_window(right=0), rows, 4, start, q, q.stride(0), 128, lse, w_in, w_out)
    ok()
    for a, b in zip((c.k, c.v, c.w), before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for s, n in enumerate(lengths):
        assert torch.equal(c.get(out, s, n), c.get(c.w, s, n))
        pages, places = c.at(s, np.arange(n))
        out[pages, :, places] = 5.0
    assert (out == 5.0).all()


def test_the_most_sequences():
    n = 1024
    lengths, new = [1 + s % 37 for s in range(n)], [(s % 3 != 1) * 1 for s in range(n)]
    c = Paged(lengths, 1, 16, 4)
    q = draw(sum(new), 2, torch.Generator().manual_seed(1))
    start = starts(new)
    o, lse = run_cached(c, dict(right=0), q, start, 2)
    weights = torch.zeros_like(c.w)
    h3.h3_cache_weights(c.cache, h3.make_window(right=0), sum(new), 2, start, q, q.stride(0), 128, lse, None, weights)
    ok()
    check_cached(c, dict(right=0), q, new, 2, o, lse, "1024 sequences")
    for s in range(n):
        # each new row's probabilities of two heads sum to 2, within a few roundings of 37 terms
        assert abs(float(c.get(weights, s, lengths[s]).double().sum()) - 2.0 * new[s]) <= 2.0 ** -16


def test_a_captured_call_follows_table_lengths_and_rows():
    """Captured with one set of sequences in a table wider than they need, replayed with others."""
    H, Hk, page, rows, width = 4, 2, 32, 120, 80
    w = h3.make_window(left=600, right=0, n_first=9)
    settings = [([500, 64, 2000], [100, 4, 16]), ([33, 2500, 10], [0, 120, 0]), ([2560, 0, 700], [1, 0, 1])]
    g = torch.Generator().manual_seed(3)
    pool = [torch.randn(110, Hk, page, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    first_weights = torch.rand(110, Hk, page, generator=g).cuda()
    q, k, v = draw(rows, H, g), draw(rows, Hk, g), draw(rows, Hk, g)
    table = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    length, start = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    kp, vp, weights = pool[0].clone(), pool[1].clone(), first_weights.clone()
    cache = h3.make_cache(kp, vp, table, length)
    o, lse = torch.empty(rows, H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, rows, device="cuda")
    ws = ws_of(h3.h3_attention_cached_workspace_bytes(cache, rows, H))
    budget = 300
    to_table = torch.arange(3 * 10, dtype=torch.int32, device="cuda").view(3, 10).flip(1).contiguous()
    tk, tv = torch.zeros(30, Hk, page, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(30, Hk, page, 128,
                                                                                             dtype=torch.bfloat16, device="cuda")
    tw, kept = torch.zeros(30, Hk, page, device="cuda"), torch.zeros(3, Hk, budget, dtype=torch.int32, device="cuda")
    to = h3.make_cache(tk, tv, to_table, torch.zeros(3, dtype=torch.int32, device="cuda"))

    def run():
        h3.h3_cache_append(cache, rows, start, k, v, k.stride(0), 128, weights)
        h3.h3_attention_cached(cache, w, rows, H, start, q, q.stride(0), 128, o, lse, ws)
        h3.h3_cache_weights(cache, w, rows, H, start, q, q.stride(0), 128, lse, weights, weights)
        h3.h3_cache_evict(cache, to, budget, 9, 100, weights, tw, kept, to._tensors[3])

    outs = [kp, vp, weights, o, lse, tk, tv, tw, kept, to._tensors[3]]

    def set_to(i, seed):
        lengths, new = settings[i]
        order, at = torch.randperm(110, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda(), 0
        table.fill_(-1)
        for s, n in enumerate(lengths):
            need = -(-n // page)
            table[s, :need] = order[at:at + need]
            at += need
        length.copy_(torch.tensor(lengths, dtype=torch.int32))
        start.copy_(starts(new))
        kp.copy_(pool[0]), vp.copy_(pool[1]), weights.copy_(first_weights)
        for t in (o, lse, tk, tv, tw, kept):
            t.zero_()

    want = []
    for i in range(3):
        set_to(i, i)
        run()
        ok()
        want.append([t.clone() for t in outs])
    graph = torch.cuda.CUDAGraph()
    set_to(0, 0)
    with torch.cuda.graph(graph):
        run()
    for i in (0, 1, 2, 1, 0):
        set_to(i, i)
        graph.replay()
        ok()
        for t, r in zip(outs, want[i]):
            assert torch.equal(t.view(torch.uint8), r.view(torch.uint8)), i
    # and what the last setting left is right
    i, (lengths, new) = 2, settings[2]
    set_to(i, i)
    run()
    ok()
    for s, n in enumerate(lengths):
        if not new[s]:
            continue
        at = sum(new[:s])
        slots = np.arange(n)
        pages, places = table[s][torch.from_numpy(slots // page).cuda()].long(), torch.from_numpy(slots % page).cuda()
        mask = O.visible(np.arange(n - new[s], n), n, left=600, right=0, n_first=9)
        for h in range(H):
            (ro, rl), (bo, bl) = O.forward(f64(q[at:at + new[s], h]), f64(kp[pages, h // 2, places]),
                                           f64(vp[pages, h // 2, places]), mask)
            within(o.view(rows, H, 128)[at:at + new[s], h], ro, bo, f"sequence {s} head {h}")
            within(lse[h, at:at + new[s]], rl, bl, f"sequence {s} head {h} lse")


def test_offsets_past_32_bits():
    """q, o and their gradients of more than 2^31 elements; the last rows of the document, which nothing before them
    changes, as a document of their own."""
    S, H, last = 131200, 128, 500
    w = dict(left=200, right=0)
    g = torch.Generator(device="cuda").manual_seed(3)
    q, d_o = (torch.randn(S, H, 128, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    k, v = (torch.randn(S, 1, 128, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    assert q.numel() > 2 ** 31
    o, lse = torch.empty(S, H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, S, device="cuda")
    window = h3.make_window(**w)
    h3.h3_attention_window(window, S, H, 1, q, H * 128, 128, k, v, 128, 128, o, lse,
                           ws_of(h3.h3_attention_window_workspace_bytes(S, H, 1)))
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    h3.h3_attention_window_backward(window, S, H, 1, q, H * 128, 128, k, v, 128, 128, o, d_o, lse, dq, H * 128, 128, dk,
                                    dv, 128, 128, ws_of(h3.h3_attention_window_backward_workspace_bytes(S, H, 1)))
    ok()
    o = o.view(S, H, 128)
    mask = O.visible(np.arange(last), last, **w)
    end = slice(S - last, S)
    sure = slice(w["left"], last)                 # rows that see nothing before the end's first, and keys only it sees
    kk, vv = f64(k[end, 0]), f64(v[end, 0])
    # outside `sure`, the end's rows miss what they saw before it: their given output is taken as it is
    for h in (0, 1, 63, 126, 127):
        (ro, rl), (bo, bl) = O.forward(f64(q[end, h]), kk, vv, mask)
        within(o[end, h][sure], ro[sure], bo[sure], f"head {h} o")
        within(lse[h, end][sure], rl[sure], bl[sure], f"head {h} lse")
    heads = range(H)
    (rq, rk, rv), (bq, bk, bv) = O.backward([f64(q[end, h]) for h in heads], kk, vv, [f64(o[end, h]) for h in heads],
                                            [f64(d_o[end, h]) for h in heads], [f64(lse[h, end]) for h in heads], mask)
    for h in (0, 1, 63, 126, 127):
        within(dq[end, h][sure], rq[h][sure], bq[h][sure], f"head {h} dq")
    within(dk[end, 0][sure], rk[sure], bk[sure], "dk")
    within(dv[end, 0][sure], rv[sure], bv[sure], "dv")
