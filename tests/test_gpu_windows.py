"""Attention in windows and over a paged cache on the GPU against the fp64 oracle (oracle/h3_window_oracle.py): every
element within the bound that its own roundings give; eviction exactly."""
import numpy as np
import pytest
import torch

import audio_video_flow_gb300 as h3
from oracle import h3_window_oracle as O

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def within(got, ref, bound, what):
    got = f64(got) if torch.is_tensor(got) else got
    assert np.isfinite(got).all(), f"{what}: not finite"
    e = np.abs(got - ref)
    worst = float((e / np.maximum(bound, 1e-45)).max()) if e.size else 0.0
    assert (e <= bound).all(), f"{what}: error {worst:.3g} times its bound"


def ok(status=0):
    torch.cuda.synchronize()
    assert h3.h3_sync_check(timeout_ms=60000) == status


def ws_of(n):
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")     # NaN wherever it is read before it is written


def draw(rows, heads, g, std=1.0, gap=0):
    """[rows][heads][128] bf16 with `gap` NaN channels behind each head."""
    t = torch.full((rows, heads, 128 + gap), float("nan"), dtype=torch.bfloat16)
    t[..., :128] = (std * torch.randn(rows, heads, 128, generator=g)).to(torch.bfloat16)
    return t.cuda()[..., :128]


def window_case(S, H, Hk, seed, std=1.0, gap=0):
    g = torch.Generator().manual_seed(seed)
    return draw(S, H, g, std, gap), draw(S, Hk, g, std, gap), draw(S, Hk, g, 1.0, gap)


def run_window(w, q, k, v, stream=None):
    S, H, Hk = q.shape[0], q.shape[1], k.shape[1]
    o = torch.full((S, H * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, S), 7.0, device="cuda")
    h3.h3_attention_window(h3.make_window(**w), S, H, Hk, q, q.stride(0), q.stride(1), k, v, k.stride(0), k.stride(1), o,
                           lse, ws_of(h3.h3_attention_window_workspace_bytes(S, H, Hk)), stream)
    return o.view(S, H, 128), lse


def check_window(w, q, k, v, o, lse, what, rows=None):
    S, H, Hk = q.shape[0], q.shape[1], k.shape[1]
    rows = np.arange(S) if rows is None else rows
    mask = O.visible(rows, S, **w)
    for h in range(H):
        (ro, rl), (bo, bl) = O.forward(f64(q[rows, h]), f64(k[:, h * Hk // H]), f64(v[:, h * Hk // H]), mask)
        within(o[rows, h], ro, bo, f"{what} head {h} o")
        within(lse[h][rows], rl, bl, f"{what} head {h} lse")


WINDOWS = [
    dict(),
    dict(left=0, right=0),
    dict(right=0),
    dict(left=-1, right=0, unit=60, origin=17),
    dict(left=1, right=0, n_first=8, unit=16, origin=8),
    dict(left=100, right=3, n_first=5),
    dict(left=0, right=0, n_first=200, unit=7, origin=3),
    dict(left=2, right=1, n_first=130, unit=33, origin=100),
    dict(left=0, right=-1, n_first=1, unit=5),
    dict(left=2147483647, right=2147483647, n_first=2147483647, unit=2147483647, origin=2147483647),
]


@pytest.mark.parametrize("w", WINDOWS, ids=lambda w: "-".join(f"{k[0]}{v}" for k, v in w.items()) or "all")
@pytest.mark.parametrize("S", [1, 5, 127, 129, 300, 601])
def test_window_forward(S, w):
    q, k, v = window_case(S, 2, 2, S)
    o, lse = run_window(w, q, k, v)
    ok()
    check_window(w, q, k, v, o, lse, f"S={S} {w}")


@pytest.mark.parametrize("S, H, Hk, gap", [(72, 4, 2, 8), (200, 6, 2, 0), (130, 7, 1, 40), (45, 8, 4, 0), (300, 5, 5, 8),
                                           (33, 128, 1, 0), (9, 100, 1, 0), (513, 16, 2, 0)])
def test_window_forward_shared_heads(S, H, Hk, gap):
    w = dict(left=70, right=0, n_first=3)
    q, k, v = window_case(S, H, Hk, S + H, gap=gap)
    o, lse = run_window(w, q, k, v)
    ok()
    check_window(w, q, k, v, o, lse, f"S={S} H={H}/{Hk}")


@pytest.mark.parametrize("H, Hk", [(1, 1), (3, 1), (57, 57)])
def test_window_forward_splits(H, Hk):
    """Few units over all SMs (each in many pieces), and more heads than shares come out even for."""
    w = dict(left=900, right=0, n_first=40)
    q, k, v = window_case(2500, H, Hk, H)
    o, lse = run_window(w, q, k, v)
    ok()
    rows = np.concatenate([np.arange(0, 2500, 61), [127, 128, 255, 256, 2499]])
    check_window(w, q, k, v, o, lse, f"H={H}", rows)


@pytest.mark.parametrize("std", [0.0, 3.0, 8.0])
def test_window_forward_flat_and_peaked(std):
    w = dict(left=3, right=0, n_first=20, unit=50)
    q, k, v = window_case(400, 2, 1, 3, std=std)
    o, lse = run_window(w, q, k, v)
    ok()
    check_window(w, q, k, v, o, lse, f"std={std}")


def test_window_everything_equals_full_attention():
    """Without bounds the window form is the document's full attention, within both calls' roundings."""
    q, k, v = window_case(505, 3, 3, 11)
    o, lse = run_window({}, q, k, v)
    qkv = torch.stack([q, k, v], dim=2).contiguous()
    full, full_lse = torch.empty(505, 3 * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 505, device="cuda")
    h3.h3_attention(505, 3, qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2], qkv.stride(0), qkv.stride(1), full, full_lse)
    ok()
    check_window({}, q, k, v, o, lse, "window")
    check_window({}, q, k, v, full.view(505, 3, 128), full_lse, "full")


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------

def backward_inputs(w, q, k, v, g):
    S, H, Hk = q.shape[0], q.shape[1], k.shape[1]
    mask = O.visible(np.arange(S), S, **w)
    o, lse = torch.empty(S, H, 128, dtype=torch.bfloat16), torch.empty(H, S)
    for h in range(H):
        (ro, rl), _ = O.forward(f64(q[:, h]), f64(k[:, h * Hk // H]), f64(v[:, h * Hk // H]), mask)
        o[:, h], lse[h] = torch.from_numpy(ro).to(torch.bfloat16), torch.from_numpy(rl).float()
    d_o = torch.randn(S, H, 128, generator=g).to(torch.bfloat16)
    return o.cuda(), lse.cuda(), d_o.cuda()


def run_backward(w, q, k, v, o, lse, d_o, gap=0, stream=None):
    S, H, Hk = q.shape[0], q.shape[1], k.shape[1]
    full = [torch.full((S, n, 128 + gap), 7.0, dtype=torch.bfloat16, device="cuda") for n in (H, Hk, Hk)]
    dq, dk, dv = (t[..., :128] for t in full)
    h3.h3_attention_window_backward(h3.make_window(**w), S, H, Hk, q, q.stride(0), q.stride(1), k, v, k.stride(0),
                                    k.stride(1), o, d_o, lse, dq, dq.stride(0), dq.stride(1), dk, dv, dk.stride(0),
                                    dk.stride(1), ws_of(h3.h3_attention_window_backward_workspace_bytes(S, H, Hk)), stream)
    for t in full:
        assert (t[..., 128:] == 7.0).all()
    return dq, dk, dv


def check_backward(w, q, k, v, o, lse, d_o, grads, what):
    S, H, Hk = q.shape[0], q.shape[1], k.shape[1]
    G = H // Hk
    mask = O.visible(np.arange(S), S, **w)
    for c in range(Hk):
        heads = range(c * G, (c + 1) * G)
        (rq, rk, rv), (bq, bk, bv) = O.backward([f64(q[:, h]) for h in heads], f64(k[:, c]), f64(v[:, c]),
                                                [f64(o[:, h]) for h in heads], [f64(d_o[:, h]) for h in heads],
                                                [f64(lse[h]) for h in heads], mask)
        for i, h in enumerate(heads):
            within(grads[0][:, h], rq[i], bq[i], f"{what} head {h} dq")
        within(grads[1][:, c], rk, bk, f"{what} kv head {c} dk")
        within(grads[2][:, c], rv, bv, f"{what} kv head {c} dv")


@pytest.mark.parametrize("w", WINDOWS, ids=lambda w: "-".join(f"{k[0]}{v}" for k, v in w.items()) or "all")
@pytest.mark.parametrize("S", [1, 5, 129, 300, 601])
def test_window_backward(S, w):
    q, k, v = window_case(S, 2, 2, S + 1)
    args = (w, q, k, v, *backward_inputs(w, q, k, v, torch.Generator().manual_seed(S)))
    grads = run_backward(*args)
    ok()
    check_backward(*args, grads, f"S={S} {w}")


@pytest.mark.parametrize("S, H, Hk, gap", [(72, 4, 2, 8), (257, 6, 2, 0), (130, 7, 1, 40), (300, 5, 5, 8), (45, 40, 1, 0)])
def test_window_backward_shared_heads(S, H, Hk, gap):
    w = dict(left=70, right=9, n_first=3)
    q, k, v = window_case(S, H, Hk, S + H, gap=gap)
    args = (w, q, k, v, *backward_inputs(w, q, k, v, torch.Generator().manual_seed(S)))
    grads = run_backward(*args, gap=gap)
    ok()
    check_backward(*args, grads, f"S={S} H={H}/{Hk}")


def test_window_backward_against_differences():
    """The gradient of sum(o * d_o) along a direction, from the forward kernel's own log-sum-exp (fp32): with
    F = sum over rows of lse, dF/dq_i = sum_j P_ij k_j / sqrt(128), which is dq for dP = 1, D = 0: here through the
    pieces that the kernel returns, by central differences of the fp64 forward."""
    w = dict(left=2, right=0, n_first=9, unit=20, origin=9)
    q, k, v = window_case(150, 2, 1, 77)
    o, lse, d_o = backward_inputs(w, q, k, v, torch.Generator().manual_seed(4))
    grads = run_backward(w, q, k, v, o, lse, d_o)
    ok()
    mask = O.visible(np.arange(150), 150, **w)
    rng = np.random.default_rng(5)
    step = 1e-4

    def loss(qq, kk, vv):
        return sum((O.forward(qq[:, h], kk[:, 0], vv[:, 0], mask)[0][0] * f64(d_o[:, h])).sum() for h in range(2))
    base = [f64(q), f64(k), f64(v)]
    for which, name in enumerate(("q", "k", "v")):
        d = rng.standard_normal(base[which].shape)
        up = [b + step * d if i == which else b for i, b in enumerate(base)]
        down = [b - step * d if i == which else b for i, b in enumerate(base)]
        slope = (loss(*up) - loss(*down)) / (2 * step)
        got = (f64(grads[which]) * d).sum()
        # rounding of P, dS and the results (2^-8 each, o's rounding in D as well), independent: relative to the
        # norm of the products 4 * 2^-8; the difference itself is good to step^2
        scale = np.sqrt(((f64(grads[which]) * d) ** 2).sum())
        assert abs(got - slope) <= 4 * 2.0 ** -8 * scale * 4, (name, got, slope, scale)


# ---------------------------------------------------------------------------
# the paged cache
# ---------------------------------------------------------------------------

class Paged:
    """Sequences of `lengths` slots in pages of a shuffled pool whose unused parts are NaN."""

    def __init__(self, lengths, heads, page, seed, extra=3, width=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lengths]
        self.page, self.heads, self.lengths = page, heads, lengths
        self.n_pages = sum(need) + extra
        order = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        width = max(max(need), 1) if width is None else width
        table = torch.full((len(lengths), width), -5, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = order[at:at + n]
            at += n
        self.host_table = table.numpy().copy()
        self.table = table.cuda()
        self.length = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        shape = (self.n_pages, heads, page, 128)
        self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        self.w = torch.full(shape[:3], 7.0, device="cuda")
        self.data = []
        for s, n in enumerate(lengths):
            k, v = draw(n, heads, g), draw(n, heads, g)
            w = torch.empty(n, heads).exponential_(generator=g).cuda()
            self.put(s, 0, k, v, w)
            self.data.append((k, v, w))
        self.cache = h3.make_cache(self.k, self.v, self.table, self.length)

    def at(self, s, slots):
        return torch.as_tensor(self.host_table[s][np.asarray(slots) // self.page].astype(np.int64)).cuda(), \
            torch.as_tensor(np.asarray(slots) % self.page).cuda()

    def put(self, s, first, k, v, w):
        pages, places = self.at(s, np.arange(first, first + len(k)))
        self.k[pages, :, places] = k
        self.v[pages, :, places] = v
        self.w[pages, :, places] = w

    def get(self, pool, s, n):
        pages, places = self.at(s, np.arange(n))
        return pool[pages, :, places]


def starts(new, lead=0):
    return torch.tensor(np.concatenate([[lead], lead + np.cumsum(new)]).astype(np.int32), device="cuda")


def run_cached(c, w, q, start, H, stream=None):
    rows = q.shape[0]
    o = torch.full((rows, H * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, rows), 7.0, device="cuda")
    h3.h3_attention_cached(c.cache, h3.make_window(**w), rows, H, start, q, q.stride(0), q.stride(1), o, lse,
                           ws_of(h3.h3_attention_cached_workspace_bytes(c.cache, rows, H)), stream)
    return o.view(rows, H, 128), lse


def check_cached(c, w, q, new, H, o, lse, what, lead=0):
    row = lead
    G = H // c.heads
    for s, n in enumerate(new):
        if n:
            k, v, _ = c.data[s]
            mask = O.visible(np.arange(c.lengths[s] - n, c.lengths[s]), c.lengths[s], **w)
            for h in range(H):
                (ro, rl), (bo, bl) = O.forward(f64(q[row:row + n, h]), f64(k[:, h // G]), f64(v[:, h // G]), mask)
                within(o[row:row + n, h], ro, bo, f"{what} sequence {s} head {h} o")
                within(lse[h, row:row + n], rl, bl, f"{what} sequence {s} head {h} lse")
        row += n


CACHED = [
    # lengths, new rows, heads, kv heads, page, window
    ([1], [1], 1, 1, 16, dict()),
    ([300], [1], 4, 4, 16, dict(right=0)),
    ([1000, 17, 128, 129, 500], [1, 1, 1, 1, 1], 8, 2, 32, dict(right=0)),
    ([1000, 17, 128, 129, 500], [1, 0, 1, 0, 1], 6, 2, 64, dict(left=40, right=0, n_first=4)),
    ([700, 333], [200, 333], 4, 2, 128, dict(right=0)),
    ([700, 333, 90], [77, 5, 90], 3, 1, 256, dict(left=1, right=0, n_first=20, unit=33, origin=20)),
    ([2000], [405], 2, 2, 16, dict(left=2, right=0, n_first=100, unit=405, origin=100)),
    ([40, 0, 3], [2, 0, 3], 7, 1, 16, dict(left=1, right=0)),
    ([4000], [2], 2, 2, 16, dict(left=0, right=0, n_first=3)),
    ([3000], [1], 56, 56, 64, dict(left=-1, right=0)),
    ([600] * 40, [1] * 40, 4, 1, 32, dict(left=500, right=0, n_first=4)),
    ([513], [257], 1, 1, 16, dict(left=10, right=5, n_first=0)),
    ([100] * 150, [1, 0, 2] * 50, 2, 1, 16, dict(right=0)),
]


@pytest.mark.parametrize("lengths, new, H, Hk, page, w", CACHED)
def test_cached_attention(lengths, new, H, Hk, page, w):
    c = Paged(lengths, Hk, page, sum(lengths))
    g = torch.Generator().manual_seed(9)
    lead, behind = 3, 5                           # rows of no sequence before the first and behind the last
    q = draw(lead + sum(new) + behind, H, g, gap=8)
    start = starts(new, lead)
    o, lse = run_cached(c, w, q, start, H)
    ok()
    check_cached(c, w, q, new, H, o, lse, f"{lengths}", lead)
    for t in (o[:lead], o[lead + sum(new):], lse[:, :lead], lse[:, lead + sum(new):]):
        assert (t == 7.0).all()


def test_cached_attention_of_a_long_cache():
    """One row over 20,000 slots: pieces on every SM."""
    c = Paged([20000], 2, 64, 5)
    q = draw(1, 4, torch.Generator().manual_seed(1))
    o, lse = run_cached(c, dict(right=0), q, starts([1]), 4)
    ok()
    check_cached(c, dict(right=0), q, [1], 4, o, lse, "long")


def test_pages_behind_the_window_are_not_looked_at():
    """Pages that no row sees may be given back: their table entries are out of range here."""
    w = dict(left=50, right=0, n_first=20)
    c = Paged([1000], 2, 16, 8)
    q = draw(3, 2, torch.Generator().manual_seed(2))
    table = c.table.clone()
    table[0, 2:59] = 1 << 30                      # slots 32 .. 943; the rows at 997 .. 999 see 947 .. and 0 .. 19
    c.cache = h3.make_cache(c.k, c.v, table, c.length)
    o, lse = run_cached(c, w, q, starts([3]), 2)
    ok()
    check_cached(c, w, q, [3], 2, o, lse, "window")


def test_append_and_attend():
    """New rows appear in their slots, the weights of those slots start at zero, nothing else changes, and the
    attention after it sees them."""
    lengths, new = [300, 40, 7], [100, 1, 7]
    c = Paged(lengths, 2, 32, 21)
    g = torch.Generator().manual_seed(3)
    k, v = draw(sum(new) + 4, 2, g, gap=8), draw(sum(new) + 4, 2, g, gap=8)
    before = [t.clone() for t in (c.k, c.v, c.w)]
    start = starts(new)
    h3.h3_cache_append(c.cache, k.shape[0], start, k, v, k.stride(0), k.stride(1), c.w)
    ok()
    row = 0
    for s, n in enumerate(new):
        pages, places = c.at(s, np.arange(lengths[s] - n, lengths[s]))
        for pool, old, rows in ((c.k, before[0], k), (c.v, before[1], v)):
            assert torch.equal(pool[pages, :, places], rows[row:row + n])
            old[pages, :, places] = rows[row:row + n]
        before[2][pages, :, places] = 0.0
        c.data[s] = (torch.cat([c.data[s][0][:-n], k[row:row + n]]), torch.cat([c.data[s][1][:-n], v[row:row + n]]), None)
        row += n
    for pool, old in zip((c.k, c.v, c.w), before):
        assert torch.equal(pool.view(torch.uint8), old.view(torch.uint8))
    q = draw(sum(new), 4, g)
    o, lse = run_cached(c, dict(right=0), q, start, 4)
    ok()
    check_cached(c, dict(right=0), q, new, 4, o, lse, "appended")


@pytest.mark.parametrize("lengths, new, H, Hk, page, w", CACHED)
def test_collected_weights(lengths, new, H, Hk, page, w):
    c = Paged(lengths, Hk, page, sum(lengths) + 1)
    q = draw(sum(new) + 2, H, torch.Generator().manual_seed(4))
    start = starts(new)
    rows = q.shape[0]
    lse = torch.full((H, rows), float("nan"), device="cuda")
    row, masks = 0, []
    for s, n in enumerate(new):
        mask = O.visible(np.arange(c.lengths[s] - n, c.lengths[s]), c.lengths[s], **w)
        masks.append(mask)
        for h in range(H if n else 0):
            (_, rl), _ = O.forward(f64(q[row:row + n, h]), f64(c.data[s][0][:, h * Hk // H]),
                                   f64(c.data[s][1][:, h * Hk // H]), mask)
            lse[h, row:row + n] = torch.from_numpy(rl).float().cuda()
        row += n
    out = torch.full_like(c.w, 5.0)
    h3.h3_cache_weights(c.cache, h3.make_window(**w), rows, H, start, q, q.stride(0), q.stride(1), lse, c.w, out)
    zero = c.w.clone()
    h3.h3_cache_weights(c.cache, h3.make_window(**w), rows, H, start, q, q.stride(0), q.stride(1), lse, None, zero)
    same = c.w.clone()
    h3.h3_cache_weights(c.cache, h3.make_window(**w), rows, H, start, q, q.stride(0), q.stride(1), lse, same, same)
    ok()
    row, used = 0, torch.zeros_like(c.w, dtype=torch.bool)
    for s, n in enumerate(new):
        length = c.lengths[s]
        pages, places = c.at(s, np.arange(length))
        used[pages, :, places] = True
        for a in range(Hk):
            heads = range(a * H // Hk, (a + 1) * H // Hk)
            ref, bound = np.zeros(length), np.zeros(length)
            if n:
                ref, bound = O.collected([f64(q[row:row + n, h]) for h in heads], f64(c.data[s][0][:, a]),
                                         [f64(lse[h, row:row + n]) for h in heads], masks[s])
            old = f64(c.get(c.w, s, length)[:, a])
            within(c.get(zero, s, length)[:, a], ref, bound + 1e-38, f"sequence {s} head {a}")
            within(c.get(out, s, length)[:, a], old + ref, bound + 2 * O.U32 * (old + ref), f"sequence {s} head {a} added")
        row += n
    assert torch.equal(same[used], out[used])
    assert (out[~used] == 5.0).all() and torch.equal(same[~used], c.w[~used])


@pytest.mark.parametrize("lengths, heads, page, budget, first, recent", [
    ([100], 1, 16, 40, 0, 0), ([100], 2, 16, 40, 4, 36), ([100, 41, 40, 39, 1, 0], 3, 16, 40, 5, 7),
    ([1111, 700, 20], 2, 32, 700, 4, 64), ([5000], 2, 128, 4999, 1, 1), ([3000], 1, 256, 1, 0, 0),
    ([2049, 2048], 1, 64, 1024, 1024, 0), ([60000], 1, 256, 20000, 100, 100)])
@pytest.mark.parametrize("kind", ["drawn", "equal", "few", "odd"])
def test_evict(lengths, heads, page, budget, first, recent, kind):
    c = Paged(lengths, heads, page, sum(lengths))
    g = torch.Generator().manual_seed(6)
    for s, n in enumerate(lengths):
        w = torch.empty(n, heads).exponential_(generator=g)
        if kind == "equal":
            w.fill_(0.25)
        elif kind == "few":                       # three values: ties everywhere
            w = torch.randint(0, 3, (n, heads), generator=g).float()
        elif kind == "odd":                       # signs, zeros of both, infinities and NaN
            w = torch.randn(n, heads, generator=g)
            pick = torch.randint(0, 12, (n, heads), generator=g)
            for i, x in enumerate((0.0, -0.0, float("inf"), float("-inf"), float("nan"))):
                w[pick == i] = x
        c.put(s, 0, c.data[s][0], c.data[s][1], w.cuda())
        c.data[s] = (c.data[s][0], c.data[s][1], w.cuda())
    to = Paged([min(n, budget) for n in lengths], heads, page, 99)
    for t, x in ((to.k, 3.0), (to.v, 3.0), (to.w, 3.0)):
        t.fill_(x)
    kept = torch.full((len(lengths), heads, budget), 77, dtype=torch.int32, device="cuda")
    length = torch.full((len(lengths),), 77, dtype=torch.int32, device="cuda")
    h3.h3_cache_evict(c.cache, h3.make_cache(to.k, to.v, to.table, length), budget, first, recent, c.w, to.w, kept, length)
    ok()
    assert length.tolist() == [min(n, budget) for n in lengths]
    used = torch.zeros_like(to.w, dtype=torch.bool)
    for s, n in enumerate(lengths):
        many = min(n, budget)
        pages, places = to.at(s, np.arange(many))
        used[pages, :, places] = True
        for h in range(heads):
            want = O.kept_slots(c.data[s][2][:, h].cpu().numpy(), budget, first, recent)
            got = kept[s, h].cpu().numpy()
            assert np.array_equal(got[:many], want) and (got[many:] == -1).all(), (s, h)
            rows = torch.from_numpy(want).cuda()
            for pool, source in ((to.k, c.data[s][0]), (to.v, c.data[s][1])):
                assert torch.equal(pool[pages, h, places], source[rows, h])
            moved, old = to.w[pages, h, places], c.data[s][2][rows, h]
            assert torch.equal(moved.view(torch.int32), old.view(torch.int32))
    assert (to.w[~used] == 3.0).all() and (to.k[~used] == 3.0).all() and (to.v[~used] == 3.0).all()


@pytest.mark.parametrize("S, H, Hk, w", [
    (2600, 2, 1, dict(left=100, right=0, n_first=5)),             # key tile 0 is seen by every row: split alone
    (2600, 4, 1, dict(right=0)),                                  # later key tiles have fewer steps than pieces
    (1500, 8, 1, dict(left=40, right=40, n_first=300)),
    (3000, 1, 1, dict(left=-1, right=0, unit=700, origin=50))])
def test_window_backward_split_key_tiles(S, H, Hk, w):
    """Key tiles whose steps are shared out over several CTAs, and joined."""
    q, k, v = window_case(S, H, Hk, S + H)
    args = (w, q, k, v, *backward_inputs(w, q, k, v, torch.Generator().manual_seed(S)))
    grads = run_backward(*args)
    ok()
    check_backward(*args, grads, f"S={S} H={H}/{Hk}")
