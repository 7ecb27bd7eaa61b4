"""Pages that a window has left behind and that another sequence has taken: the old entries of the first sequence's table
still name them."""
import numpy as np
import pytest
import torch

import audio_video_flow_gb300 as h3
from oracle import h3_window_oracle as O
from test_gpu_windows import Paged, draw, f64, ok, run_cached, starts, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new, H, Hk, page", [([200, 1], 4, 2, 16), ([3, 40], 2, 2, 64), ([1, 1], 8, 1, 32),
                                              ([405, 1], 40, 40, 16)])
def test_pages_that_another_sequence_took(new, H, Hk, page):
    """Attention does not look at them, and weights collected in place leave them to their new owner."""
    w = dict(left=50, right=0, n_first=20)
    n = 1280
    # no row of the first sequence sees these pages' slots
    free = np.arange(-(-20 // page), (n - new[0] - 50) // page)
    lengths = [n, len(free) * page]
    c = Paged(lengths, Hk, page, 8)
    g = torch.Generator().manual_seed(2)
    q = draw(sum(new), H, g)
    start = starts(new)
    clean, stale = c.table.clone(), c.table.clone()
    clean[0, torch.from_numpy(free).cuda()] = -5
    stale[0, torch.from_numpy(free).cuda()] = c.table[1, :len(free)]
    caches = [h3.make_cache(c.k, c.v, t, c.length) for t in (clean, stale)]
    runs = []
    for cache in caches:
        c.cache = cache
        runs.append(run_cached(c, w, q, start, H))
    ok()
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    lse = runs[0][1]
    weights = []
    for i, cache in enumerate([caches[0]] + [caches[1]] * 20):
        weights.append(c.w.clone())
        h3.h3_cache_weights(cache, h3.make_window(**w), sum(new), H, start, q, q.stride(0), q.stride(1), lse, weights[-1],
                            weights[-1])
    ok()
    for t in weights[1:]:
        assert torch.equal(t.view(torch.int32), weights[0].view(torch.int32))
    row = 0
    for s, many in enumerate(new):
        mask = O.visible(np.arange(lengths[s] - many, lengths[s]), lengths[s], **w)
        seen = np.flatnonzero(mask.any(axis=0))
        pages, places = c.at(s, seen)
        for a in range(Hk):
            heads = range(a * H // Hk, (a + 1) * H // Hk)
            ref, bound = O.collected([f64(q[row:row + many, h]) for h in heads], f64(c.data[s][0][:, a]),
                                     [f64(lse[h, row:row + many]) for h in heads], mask)
            total = f64(c.data[s][2][:, a])[seen] + ref[seen]
            within(weights[0][pages, a, places], total, bound[seen] + 2 * O.U32 * total, f"sequence {s} head {a}")
        row += many
    used = torch.zeros_like(c.w, dtype=torch.bool)         # slots that a row sees
    row = 0
    for s, many in enumerate(new):
        mask = O.visible(np.arange(lengths[s] - many, lengths[s]), lengths[s], **w)
        pages, places = c.at(s, np.flatnonzero(mask.any(axis=0)))
        used[pages, :, places] = True
    assert torch.equal(weights[0][~used], c.w[~used])


@pytest.mark.parametrize("page, new", [(16, 200), (64, 3), (32, 1)])
def test_a_sequence_that_reuses_its_own_pages(page, new):
    """A ring: the entries of slots that the window has left name pages that newer slots of the same sequence stand in."""
    w, n, H, Hk = dict(left=50, right=0, n_first=20), 1280, 4, 2
    free = np.arange(-(-20 // page), (n - new - 50) // page)
    kept = np.arange((n - new - 50) // page, n // page)
    c = Paged([n], Hk, page, 8)
    q = draw(new, H, torch.Generator().manual_seed(2))
    start = starts([new])
    clean, ring = c.table.clone(), c.table.clone()
    clean[0, torch.from_numpy(free).cuda()] = -5
    ring[0, torch.from_numpy(free).cuda()] = c.table[0, torch.from_numpy(np.resize(kept, len(free))).cuda()]
    results = []
    for table in [clean] + [ring] * 10:
        c.cache = h3.make_cache(c.k, c.v, table, c.length)
        o, lse = run_cached(c, w, q, start, H)
        weights = c.w.clone()
        h3.h3_cache_weights(c.cache, h3.make_window(**w), new, H, start, q, q.stride(0), q.stride(1), lse, weights, weights)
        results.append((o, lse, weights))
    ok()
    for r in results[1:]:
        for a, b in zip(r, results[0]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
