"""Bad metadata of a sequence that none of a call's rows leads to: every call reports it."""
import pytest
import torch

import audio_video_flow_gb300 as h3
from test_gpu_windows import Paged, draw, ok, run_cached, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", ["long", "negative", "ends early"])
def test_a_sequence_without_rows_is_reported(what):
    lengths, new = [100, 80, 60], [10, 0, 3]
    c = Paged(lengths, 2, 16, 31)
    start = starts(new)
    good = [0, 2]
    if what == "long":
        c.length[1] = 1 << 20
    elif what == "negative":
        c.length[1] = -1
    else:
        # rows 10, 11 and 12 are the second's, and the third ends before it begins
        start = torch.tensor([0, 10, 13, 10], dtype=torch.int32, device="cuda")
        good = [0]
    rows = sum(new)
    k, v, q = (draw(rows, 2, torch.Generator().manual_seed(8 + i)) for i in range(3))
    before = [t.clone() for t in (c.k, c.v, c.w)]
    h3.h3_cache_append(c.cache, rows, start, k, v, k.stride(0), k.stride(1), c.w)
    ok(h3.H3_ERR_INDEX)
    for s in good:
        at = [0, 10, 10][s]
        for slot in range(lengths[s] - new[s], lengths[s]):
            pages, places = c.at(s, [slot])
            for pool, old, new_rows in ((c.k, before[0], k), (c.v, before[1], v)):
                assert torch.equal(pool[pages, :, places][0], new_rows[at])
                old[pages, :, places] = new_rows[at]
            before[2][pages, :, places] = 0.0
            at += 1
    if what != "ends early":                      # (its second sequence is a good one of three rows)
        for pool, old in zip((c.k, c.v, c.w), before):
            assert torch.equal(pool.view(torch.uint8), old.view(torch.uint8))
    o, lse = run_cached(c, dict(right=0), q, start, 2)
    ok(h3.H3_ERR_INDEX)
    h3.h3_cache_weights(c.cache, h3.make_window(right=0), rows, 2, start, q, q.stride(0), q.stride(1), lse, c.w, c.w)
    ok(h3.H3_ERR_INDEX)
