"""The window and cache entry points on the host: sizes of workspaces, and every refusal, which returns before anything
would be launched; and the oracle of these operators against brute force."""
import ctypes
import math

import numpy as np
import pytest

import audio_video_flow_gb300 as h3
from audio_video_flow_gb300 import _build
from oracle import h3_window_oracle as O


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return h3.lib()


def _call(f, args, **changed):
    a = dict(args)
    for k, v in changed.items():
        if "." in k:                       # a field of a struct
            name, field = k.split(".")
            c = type(a[name]).from_buffer_copy(a[name])
            setattr(c, field, v)
            a[name] = c
        else:
            a[k] = v
    return f(*[ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in a.values()])


WINDOW = h3.make_window(4, 0, 3, 16, 5)
CACHE = h3.Cache(0x10000, 0x20000, 10, 16, 2, 3, 4, 0x30000, 0x31000)
TO = h3.Cache(0x40000, 0x50000, 10, 32, 2, 3, 4, 0x60000, 0x61000)
BIG = 1 << 40

FORWARD = dict(window=WINDOW, n_rows=8, n_heads=4, n_kv_heads=2, q=0x1000, qrs=512, qhs=128, k=0x2000, v=0x3000, krs=256,
               khs=128, o=0x4000, lse=0x5000, ws=0x100000, ws_bytes=BIG, stream=None)
BACKWARD = dict(window=WINDOW, n_rows=8, n_heads=4, n_kv_heads=2, q=0x1000, qrs=512, qhs=128, k=0x2000, v=0x3000, krs=256,
                khs=128, o=0x4000, d_o=0x6000, lse=0x5000, dq=0x7000, dqrs=512, dqhs=128, dk=0x8000, dv=0x9000, dkrs=256,
                dkhs=128, ws=0x100000, ws_bytes=BIG, stream=None)
APPEND = dict(cache=CACHE, n_rows=8, start=0x1000, k=0x2000, v=0x3000, rs=256, hs=128, weights=0x4000, stream=None)
CACHED = dict(cache=CACHE, window=WINDOW, n_rows=8, n_heads=4, start=0x1000, q=0x2000, qrs=512, qhs=128, o=0x4000,
              lse=0x5000, ws=0x100000, ws_bytes=BIG, stream=None)
WEIGHTS = dict(cache=CACHE, window=WINDOW, n_rows=8, n_heads=4, start=0x1000, q=0x2000, qrs=512, qhs=128, lse=0x5000,
               w_in=0x6000, w_out=0x7000, stream=None)
EVICT = dict(cache=CACHE, to=TO, budget=20, first=4, recent=6, weights=0x1000, weights_to=0x2000, kept=0x3000,
             length=0x4000, stream=None)

BAD_WINDOWS = [({f"window.{f}": v}, h3.H3_ERR_SHAPE) for f, v in
               [("left", -2), ("right", -2), ("n_first", -1), ("unit", 0), ("unit", -5), ("origin", -1)]]
BAD_HEADS = [(dict(n_rows=0), h3.H3_ERR_SHAPE), (dict(n_rows=-3), h3.H3_ERR_SHAPE), (dict(n_heads=0), h3.H3_ERR_SHAPE),
             (dict(n_heads=5), h3.H3_ERR_SHAPE), (dict(n_heads=258), h3.H3_ERR_UNSUPPORTED),
             (dict(n_rows=(1 << 24) + 1), h3.H3_ERR_UNSUPPORTED)]
BAD_Q = [(dict(qrs=120), h3.H3_ERR_SHAPE), (dict(qhs=64), h3.H3_ERR_SHAPE), (dict(qrs=516), h3.H3_ERR_ALIGN),
         (dict(qhs=129), h3.H3_ERR_ALIGN), (dict(q=0x1008), h3.H3_ERR_ALIGN), (dict(qrs=1 << 40), h3.H3_ERR_UNSUPPORTED),
         (dict(lse=0x5002), h3.H3_ERR_ALIGN)]
BAD_CACHES = [({"cache.n_pages": 0}, h3.H3_ERR_SHAPE), ({"cache.n_kv_heads": 0}, h3.H3_ERR_SHAPE),
              ({"cache.n_seqs": 0}, h3.H3_ERR_SHAPE), ({"cache.table_width": 0}, h3.H3_ERR_SHAPE),
              ({"cache.page_size": 8}, h3.H3_ERR_UNSUPPORTED), ({"cache.page_size": 48}, h3.H3_ERR_UNSUPPORTED),
              ({"cache.page_size": 512}, h3.H3_ERR_UNSUPPORTED), ({"cache.n_seqs": 1025}, h3.H3_ERR_UNSUPPORTED),
              ({"cache.table_width": (1 << 20) + 1}, h3.H3_ERR_UNSUPPORTED), ({"cache.k": None}, h3.H3_ERR_NULL),
              ({"cache.v": None}, h3.H3_ERR_NULL), ({"cache.table": None}, h3.H3_ERR_NULL),
              ({"cache.length": None}, h3.H3_ERR_NULL), ({"cache.k": 0x10008}, h3.H3_ERR_ALIGN),
              ({"cache.table": 0x30002}, h3.H3_ERR_ALIGN), ({"cache.v": 0x10000}, h3.H3_ERR_SHAPE)]


def _ids(v):
    return str(v) if isinstance(v, dict) else None


@pytest.mark.parametrize("changed, status", BAD_WINDOWS + BAD_HEADS + BAD_Q + [
    (dict(krs=64), h3.H3_ERR_SHAPE), (dict(khs=12), h3.H3_ERR_SHAPE), (dict(krs=260), h3.H3_ERR_ALIGN),
    (dict(o=0x4008), h3.H3_ERR_ALIGN), (dict(ws=0x100010), h3.H3_ERR_ALIGN), (dict(o=0x1000), h3.H3_ERR_SHAPE),
    (dict(o=0x3000), h3.H3_ERR_SHAPE), (dict(o=0x100000), h3.H3_ERR_SHAPE), (dict(lse=0x4000), h3.H3_ERR_SHAPE),
    (dict(ws_bytes=100), h3.H3_ERR_WORKSPACE)], ids=_ids)
def test_window_refuses(lib, changed, status):
    assert _call(lib.h3_attention_window, FORWARD, **changed) == status


@pytest.mark.parametrize("changed, status", BAD_WINDOWS + BAD_HEADS + BAD_Q + [
    (dict(dqrs=120), h3.H3_ERR_SHAPE), (dict(dkhs=132), h3.H3_ERR_ALIGN), (dict(dqrs=128), h3.H3_ERR_SHAPE),
    (dict(dkrs=128), h3.H3_ERR_SHAPE), (dict(dv=0x9008), h3.H3_ERR_ALIGN), (dict(d_o=0x6002), h3.H3_ERR_ALIGN),
    (dict(dq=0x1000), h3.H3_ERR_SHAPE), (dict(dk=0x7000), h3.H3_ERR_SHAPE), (dict(dv=0x6000), h3.H3_ERR_SHAPE),
    (dict(ws_bytes=4095), h3.H3_ERR_WORKSPACE)], ids=_ids)
def test_window_backward_refuses(lib, changed, status):
    assert _call(lib.h3_attention_window_backward, BACKWARD, **changed) == status


@pytest.mark.parametrize("changed, status", BAD_CACHES + [
    (dict(n_rows=0), h3.H3_ERR_SHAPE), (dict(n_rows=(1 << 24) + 1), h3.H3_ERR_UNSUPPORTED), (dict(rs=120), h3.H3_ERR_SHAPE),
    (dict(hs=132), h3.H3_ERR_ALIGN), (dict(k=0x2008), h3.H3_ERR_ALIGN), (dict(start=0x1002), h3.H3_ERR_ALIGN),
    (dict(weights=0x4001), h3.H3_ERR_ALIGN), (dict(k=0x10000), h3.H3_ERR_SHAPE), (dict(v=0x10000), h3.H3_ERR_SHAPE)],
    ids=_ids)
def test_append_refuses(lib, changed, status):
    assert _call(lib.h3_cache_append, APPEND, **changed) == status


@pytest.mark.parametrize("changed, status", BAD_CACHES + BAD_WINDOWS + BAD_HEADS + BAD_Q + [
    (dict(o=0x4008), h3.H3_ERR_ALIGN), (dict(ws=0x100010), h3.H3_ERR_ALIGN), (dict(start=0x1001), h3.H3_ERR_ALIGN),
    (dict(o=0x2000), h3.H3_ERR_SHAPE), (dict(o=0x20000), h3.H3_ERR_SHAPE), (dict(lse=0x100000), h3.H3_ERR_SHAPE),
    (dict(ws_bytes=100), h3.H3_ERR_WORKSPACE)], ids=_ids)
def test_cached_refuses(lib, changed, status):
    assert _call(lib.h3_attention_cached, CACHED, **changed) == status


@pytest.mark.parametrize("changed, status", BAD_CACHES + BAD_WINDOWS + BAD_HEADS + BAD_Q + [
    (dict(w_in=0x6002), h3.H3_ERR_ALIGN), (dict(w_out=0x7002), h3.H3_ERR_ALIGN), (dict(w_out=0x5000), h3.H3_ERR_SHAPE),
    (dict(w_out=0x2000), h3.H3_ERR_SHAPE), (dict(w_out=0x10000), h3.H3_ERR_SHAPE)], ids=_ids)
def test_weights_refuses(lib, changed, status):
    assert _call(lib.h3_cache_weights, WEIGHTS, **changed) == status


@pytest.mark.parametrize("changed, status", BAD_CACHES + [
    (dict(budget=0), h3.H3_ERR_SHAPE), (dict(first=-1), h3.H3_ERR_SHAPE), (dict(recent=-1), h3.H3_ERR_SHAPE),
    (dict(first=15), h3.H3_ERR_SHAPE), (dict(first=2147483647, recent=2147483647), h3.H3_ERR_SHAPE),
    (dict(budget=(1 << 24) + 1), h3.H3_ERR_UNSUPPORTED), ({"to.n_kv_heads": 3}, h3.H3_ERR_SHAPE),
    ({"to.n_seqs": 2}, h3.H3_ERR_SHAPE), ({"to.table": 0x30000}, h3.H3_ERR_SHAPE), ({"to.k": 0x20000}, h3.H3_ERR_SHAPE),
    (dict(length=0x31000), h3.H3_ERR_SHAPE), (dict(kept=0x4000), h3.H3_ERR_SHAPE), (dict(kept=0x3002), h3.H3_ERR_ALIGN),
    (dict(weights=0x1001), h3.H3_ERR_ALIGN), ({"to.page_size": 24}, h3.H3_ERR_UNSUPPORTED)], ids=_ids)
def test_evict_refuses(lib, changed, status):
    assert _call(lib.h3_cache_evict, EVICT, **changed) == status


@pytest.mark.parametrize("f, args, names", [
    ("h3_attention_window", FORWARD, "window q k v o ws"),
    ("h3_attention_window_backward", BACKWARD, "window q k v o d_o lse dq dk dv ws"),
    ("h3_cache_append", APPEND, "cache start k v"), ("h3_attention_cached", CACHED, "cache window start q o ws"),
    ("h3_cache_weights", WEIGHTS, "cache window start q lse w_out"),
    ("h3_cache_evict", EVICT, "cache to weights kept length")])
def test_null_is_refused(lib, f, args, names):
    for name in names.split():
        assert _call(getattr(lib, f), args, **{name: None}) == h3.H3_ERR_NULL, name


def test_more_work_than_runs_can_count_is_refused(lib):
    """2^24 rows without a window are 2^33 pairs of a unit and a key tile; with one they fit."""
    assert _call(lib.h3_attention_window, FORWARD, n_rows=1 << 24, **{"window.left": -1}) == h3.H3_ERR_UNSUPPORTED
    assert _call(lib.h3_attention_window, FORWARD, n_rows=1 << 24, ws_bytes=1) == h3.H3_ERR_WORKSPACE


def test_workspaces(lib):
    f = h3.h3_attention_window_workspace_bytes
    assert 0 < f(1, 4, 2) <= f(8, 4, 2) <= f(500, 4, 2) == f(1 << 24, 4, 2)
    assert f(0, 4, 2) == f(8, 5, 2) == f(8, 258, 2) == f(-1, 4, 2) == f((1 << 24) + 1, 4, 2) == 0
    b = h3.h3_attention_window_backward_workspace_bytes
    assert b(8, 4, 2) == h3.h3_attention_backward_workspace_bytes(8, 4)
    assert b(5000, 4, 2) > h3.h3_attention_backward_workspace_bytes(5000, 4)
    assert b(8, 5, 2) == 0
    c = h3.h3_attention_cached_workspace_bytes
    assert c(CACHE, 8, 4) > 0 and c(CACHE, 8, 5) == 0
    bad = h3.Cache.from_buffer_copy(CACHE)
    bad.page_size = 17
    assert c(bad, 8, 4) == 0


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("w", [dict(), dict(left=0, right=0), dict(left=2, right=1, n_first=3, unit=4, origin=6),
                               dict(right=0), dict(left=1, n_first=9, unit=5, origin=2)])
def test_visible_against_the_definition(w):
    p = dict(left=-1, right=-1, n_first=0, unit=1, origin=0)
    p.update(w)
    seen = O.visible(np.arange(7, 30), 30, **w)
    for i in range(7, 30):
        for j in range(30):
            ui, uj = (i - p["origin"]) // p["unit"], (j - p["origin"]) // p["unit"]
            want = (p["right"] < 0 or uj <= ui + p["right"]) and \
                   (p["left"] < 0 or uj >= ui - p["left"] or j < p["n_first"])
            assert seen[i - 7, j] == want
    assert seen[np.arange(23), np.arange(7, 30)].all()


def test_forward_and_collected_against_loops():
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((n, 128)) for n in (5, 9, 9))
    mask = O.visible(np.arange(4, 9), 9, left=2, right=0, n_first=1)
    (o, lse), _ = O.forward(q, k, v, mask)
    total = np.zeros(9)
    for i in range(5):
        js = [j for j in range(9) if mask[i, j]]
        e = np.array([math.exp(q[i] @ k[j] / math.sqrt(128)) for j in js])
        assert np.allclose(o[i], sum(x * v[j] for x, j in zip(e, js)) / e.sum(), rtol=1e-12)
        assert math.isclose(lse[i], math.log(e.sum()), rel_tol=1e-12)
        total[js] += e / e.sum()
    assert np.allclose(O.collected([q], k, [lse], mask)[0], total, rtol=1e-12)


def test_backward_against_differences():
    """Two query heads over one KV head: d sum(o * d_o) by central differences."""
    rng = np.random.default_rng(4)
    qs, d_os = ([rng.standard_normal((6, 128)) for _ in range(2)] for _ in range(2))
    k, v = rng.standard_normal((6, 128)), rng.standard_normal((6, 128))
    mask = O.visible(np.arange(6), 6, left=1, right=0, n_first=1)

    def loss(qs, k, v):
        return sum((O.forward(q, k, v, mask)[0][0] * d).sum() for q, d in zip(qs, d_os))
    outs = [O.forward(q, k, v, mask)[0] for q in qs]
    (dqs, dk, dv), _ = O.backward(qs, k, v, [o for o, _ in outs], d_os, [s for _, s in outs], mask)
    h = 1e-5
    for n, (i, c) in enumerate([(0, 3), (2, 100), (5, 64), (3, 0)]):
        def moved(x, by):
            y = x.copy()
            y[i, c] += by
            return y
        slope = (loss(qs, moved(k, h), v) - loss(qs, moved(k, -h), v)) / (2 * h)
        assert math.isclose(slope, dk[i, c], rel_tol=1e-6, abs_tol=1e-8)
        slope = (loss(qs, k, moved(v, h)) - loss(qs, k, moved(v, -h))) / (2 * h)
        assert math.isclose(slope, dv[i, c], rel_tol=1e-6, abs_tol=1e-8)
        slope = (loss([moved(qs[0], h), qs[1]], k, v) - loss([moved(qs[0], -h), qs[1]], k, v)) / (2 * h)
        assert math.isclose(slope, dqs[0][i, c], rel_tol=1e-6, abs_tol=1e-8)


def test_kept_slots_against_a_plain_search():
    rng = np.random.default_rng(5)
    for n, budget, first, recent in [(10, 4, 1, 2), (10, 10, 1, 2), (30, 7, 0, 0), (9, 8, 8, 0), (12, 5, 2, 3)]:
        for values in (rng.standard_normal(n), rng.integers(0, 3, n).astype(float), np.full(n, np.nan),
                       np.where(rng.random(n) < 0.5, np.nan, -np.inf)):
            w = values.astype(np.float32)
            kept = set(range(n)) if n <= budget else set(range(first)) | set(range(n - recent, n))
            rank = lambda j: (0, 0.0) if np.isnan(w[j]) else (1, float(w[j]))  # noqa: E731
            while len(kept) < min(n, budget):
                rest = [j for j in range(first, n - recent) if j not in kept]
                best = max(rest, key=lambda j: (rank(j), -j))
                kept.add(best)
            assert list(O.kept_slots(w, budget, first, recent)) == sorted(kept)
