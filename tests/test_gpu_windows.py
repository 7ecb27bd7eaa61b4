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


# ---------------------------------------------------------------------------
# the cache in other shapes, bad metadata, streams and graphs, the operators together
# ---------------------------------------------------------------------------

def test_cached_attention_of_rows_with_one_longer_document():
    """Single rows on average, so units of one tile; one document has several."""
    lengths, new = [900] + [50] * 20, [300] + [1] * 20
    c = Paged(lengths, 1, 16, 3)
    q = draw(sum(new), 1, torch.Generator().manual_seed(3))
    w = dict(left=200, right=0, n_first=4)
    o, lse = run_cached(c, w, q, starts(new), 1)
    ok()
    check_cached(c, w, q, new, 1, o, lse, "rows")


def test_a_long_cache_of_one_head_and_a_chunk():
    """Units that every SM has a part of, of a chunk and of one row."""
    for new, H in (([200], 1), ([1], 1), ([2], 5)):
        c = Paged([12345], 1, 128, 4)
        q = draw(sum(new), H, torch.Generator().manual_seed(4))
        o, lse = run_cached(c, dict(right=0), q, starts(new), H)
        ok()
        check_cached(c, dict(right=0), q, new, H, o, lse, str(new))


def test_pages_past_32_bits():
    """A pool of more than 2^31 elements: the pages in use are its last ones."""
    n_pages, page = 8200, 256                     # x 8 heads x 128: 2.15e9 elements a pool
    g = torch.Generator().manual_seed(6)
    k = torch.empty(n_pages, 8, page, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device="cuda")
    length = torch.tensor([300], dtype=torch.int32, device="cuda")
    cache = h3.make_cache(k, v, table, length)
    kn, vn = draw(300, 8, g), draw(300, 8, g)
    start = starts([300])
    weights = torch.zeros(n_pages, 8, page, device="cuda")
    h3.h3_cache_append(cache, 300, start, kn, vn, kn.stride(0), kn.stride(1), weights)
    ok()
    for t, new in ((k, kn), (v, vn)):
        assert torch.equal(t[-1].transpose(0, 1), new[:256]) and torch.equal(t[-2, :, :44].transpose(0, 1), new[256:])
    c = Paged([1], 8, 16, 1)
    c.cache, c.lengths, c.data = cache, [300], [(kn, vn, None)]
    q = draw(300, 8, g)
    o, lse = run_cached(c, dict(right=0), q, start, 8)
    h3.h3_cache_weights(cache, h3.make_window(right=0), 300, 8, start, q, q.stride(0), q.stride(1), lse, weights, weights)
    ok()
    check_cached(c, dict(right=0), q, [300], 8, o, lse, "far pages")
    total = weights[-1].double().sum() + weights[-2].double().sum()
    # every row's probabilities sum to 1: 300 rows x 8 heads, within the sums' own rounding
    assert abs(float(total) - 2400.0) <= 2400 * 2.0 ** -16
    to = Paged([100], 8, 16, 2)
    kept = torch.empty(1, 8, 100, dtype=torch.int32, device="cuda")
    h3.h3_cache_evict(cache, to.cache, 100, 1, 1, weights, to.w, kept, to.length)
    ok()
    for h in range(8):
        w = torch.cat([weights[-1, h], weights[-2, h, :44]]).cpu().numpy()
        want = O.kept_slots(w, 100, 1, 1)
        assert np.array_equal(kept[0, h].cpu().numpy(), want)
        pages, places = to.at(0, np.arange(100))
        assert torch.equal(to.k[pages, h, places], kn[torch.from_numpy(want).cuda(), h])


@pytest.mark.parametrize("what", ["length", "short", "start", "page"])
def test_bad_metadata_is_reported(what):
    """Found on the device: the status says so, the other sequences are right, and nothing of the bad one is written
    (a bad page leaves its rows undefined)."""
    lengths, new = [100, 80, 60], [3, 2, 1]
    c = Paged(lengths, 2, 16, 31)
    q = draw(6, 2, torch.Generator().manual_seed(7))
    start = starts(new)
    if what == "length":
        c.length[1] = 1 << 20
    elif what == "short":
        c.length[1] = 1                          # fewer than its new rows
    elif what == "start":
        start[2] = 2                             # sequence 1 ends before it begins
    else:
        c.table[1, 2] = 12345
    o, lse = run_cached(c, dict(right=0), q, start, 2)
    ok(h3.H3_ERR_INDEX)
    good = [3, 0, 1] if what != "start" else [3, 0, 0]
    for s, n in enumerate(good):
        if n:
            at = [0, 3, 5][s]
            k, v, _ = c.data[s]
            mask = O.visible(np.arange(lengths[s] - n, lengths[s]), lengths[s], right=0)
            for h in range(2):
                (ro, _), (bo, _) = O.forward(f64(q[at:at + n, h]), f64(k[:, h]), f64(v[:, h]), mask)
                within(o[at:at + n, h], ro, bo, f"sequence {s}")
    if what in ("length", "short"):
        assert (o[3:5] == 7.0).all() and (lse[:, 3:5] == 7.0).all()
    before = c.k.clone()
    k = draw(6, 2, torch.Generator().manual_seed(8))
    if what != "page":                            # (new rows lie in the document's last page)
        h3.h3_cache_append(c.cache, 6, start, k, k, k.stride(0), k.stride(1))
        ok(h3.H3_ERR_INDEX)
        pages, _ = c.at(1, np.arange(80))
        assert torch.equal(c.k[pages].view(torch.int16), before[pages].view(torch.int16))
    out = torch.full_like(c.w, 5.0)
    lse = torch.zeros(2, 6, device="cuda")
    h3.h3_cache_weights(c.cache, h3.make_window(right=0), 6, 2, start, q, q.stride(0), q.stride(1), lse, c.w, out)
    ok(h3.H3_ERR_INDEX)
    if what in ("length", "page"):
        kept = torch.empty(3, 2, 20, dtype=torch.int32, device="cuda")
        to = Paged([20, 20, 20], 2, 16, 5)
        h3.h3_cache_evict(c.cache, to.cache, 20, 2, 2, c.w, to.w, kept, to.length)
        ok(h3.H3_ERR_INDEX)
        for s in (0, 2):
            for h in range(2):
                want = O.kept_slots(c.data[s][2][:, h].cpu().numpy(), 20, 2, 2)
                assert np.array_equal(kept[s, h].cpu().numpy(), want)


def calls(seed):
    """One call of each operator, ready to be made: (run(stream), its outputs)."""
    g = torch.Generator().manual_seed(seed)
    w = h3.make_window(2, 0, 17, 60, 17)
    S, H, Hk = 700, 6, 3
    q, k, v = draw(S, H, g), draw(S, Hk, g), draw(S, Hk, g)
    o, lse = torch.empty(S, H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, S, device="cuda")
    ws = ws_of(h3.h3_attention_window_workspace_bytes(S, H, Hk))
    d_o = draw(S, H, g).contiguous()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws2 = ws_of(h3.h3_attention_window_backward_workspace_bytes(S, H, Hk))
    c = Paged([1500, 40], Hk, 32, seed)
    qc, kc, vc = draw(210, H, g), draw(210, Hk, g), draw(210, Hk, g)
    start = starts([200, 10])
    oc, lc = torch.empty(210, H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, 210, device="cuda")
    ws3 = ws_of(h3.h3_attention_cached_workspace_bytes(c.cache, 210, H))
    out = c.w.clone()
    to = Paged([300, 40], Hk, 64, seed + 1)
    to.k.zero_(), to.v.zero_(), to.w.zero_()
    kept = torch.empty(2, Hk, 300, dtype=torch.int32, device="cuda")

    def run(stream=None):
        h3.h3_attention_window(w, S, H, Hk, q, q.stride(0), 128, k, v, k.stride(0), 128, o, lse, ws, stream)
        h3.h3_attention_window_backward(w, S, H, Hk, q, q.stride(0), 128, k, v, k.stride(0), 128, o, d_o, lse, dq,
                                        dq.stride(0), 128, dk, dv, dk.stride(0), 128, ws2, stream)
        h3.h3_cache_append(c.cache, 210, start, kc, vc, kc.stride(0), 128, c.w, stream)
        h3.h3_attention_cached(c.cache, w, 210, H, start, qc, qc.stride(0), 128, oc, lc, ws3, stream)
        h3.h3_cache_weights(c.cache, w, 210, H, start, qc, qc.stride(0), 128, lc, c.w, out, stream)
        h3.h3_cache_evict(c.cache, to.cache, 300, 17, 200, out, to.w, kept, to.length, stream)
    return run, [o, lse, dq, dk, dv, oc, lc, out, kept, to.k, to.v, to.w]


def test_streams_graphs_and_repeats_give_the_same_bits():
    runs = [calls(seed) for seed in (1, 2, 3)]
    want = []
    for run, outs in runs:
        run()
        ok()
        want.append([t.clone() for t in outs])
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(10):                           # several at once
        for (run, _), s in zip(runs, streams):
            run(s)
    ok()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                 # captured, and replayed beside an eager call
        runs[0][0]()
    for _ in range(5):
        graph.replay()
        runs[1][0](streams[1])
    ok()
    for (_, outs), ref in zip(runs, want):
        for t, r in zip(outs, ref):
            assert torch.equal(t.view(torch.uint8), r.view(torch.uint8))


def test_a_clip_generated_frame_by_frame():
    """Frames appended and attended to one after the other give what the window gives over the whole clip; the weights
    that they collect go by every row's probabilities; and after the cache is cut, the next frame attends to what was
    kept."""
    H, Hk, frame, text, frames = 4, 2, 45, 10, 6
    S = text + frame * frames
    w = dict(left=2, right=0, n_first=text, unit=frame, origin=text)
    g = torch.Generator().manual_seed(12)
    q, k, v = draw(S, H, g), draw(S, Hk, g), draw(S, Hk, g)
    whole, whole_lse = run_window(w, q, k, v)
    table = torch.tensor([[7, 2, 5, 0, 1, 6, 3, 4, 9, 8]], dtype=torch.int32, device="cuda")
    pools = [torch.full((10, Hk, 32, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    weights = torch.full((10, Hk, 32), float("nan"), device="cuda")
    length = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = h3.make_cache(*pools, table, length)
    window = h3.make_window(**w)
    row, total = 0, 0.0
    for n in [text] + [frame] * frames:
        part = slice(row, row + n)
        row += n
        length.fill_(row)
        start = starts([n])
        h3.h3_cache_append(cache, n, start, k[part], v[part], k.stride(0), k.stride(1), weights)
        o, lse = torch.empty(n, H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, n, device="cuda")
        h3.h3_attention_cached(cache, window, n, H, start, q[part], q.stride(0), q.stride(1), o, lse,
                               ws_of(h3.h3_attention_cached_workspace_bytes(cache, n, H)))
        h3.h3_cache_weights(cache, window, n, H, start, q[part], q.stride(0), q.stride(1), lse, weights, weights)
        ok()
        mask = O.visible(np.arange(row - n, row), S, **w)
        for h in range(H):
            (ro, rl), (bo, bl) = O.forward(f64(q[part, h]), f64(k[:, h * Hk // H]), f64(v[:, h * Hk // H]), mask)
            within(o.view(n, H, 128)[:, h], ro, bo, f"rows {part} head {h}")
            within(lse[h], rl, bl, f"rows {part} head {h} lse")
            within(whole[part, h], ro, bo, f"whole clip, rows {part} head {h}")
            within(whole_lse[h][part], rl, bl, f"whole clip, rows {part} head {h} lse")
    slots = torch.arange(S, device="cuda")
    mine = weights[table[0, slots // 32].long(), :, slots % 32]
    assert abs(float(mine.double().sum()) - S * H) <= S * H * 2.0 ** -16
    # cut to 120 rows, the text and the last frame kept
    to_table = torch.tensor([[3, 1, 4, 0, 2, 5]], dtype=torch.int32, device="cuda")
    to_pools = [torch.full((6, Hk, 32, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    to_weights = torch.full((6, Hk, 32), float("nan"), device="cuda")
    to_length = torch.zeros(1, dtype=torch.int32, device="cuda")
    to = h3.make_cache(*to_pools, to_table, to_length)
    kept = torch.empty(1, Hk, 120, dtype=torch.int32, device="cuda")
    h3.h3_cache_evict(cache, to, 120, text, frame, weights, to_weights, kept, to_length)
    ok()
    assert to_length.item() == 120
    kn, vn, qn = draw(frame, Hk, g), draw(frame, Hk, g), draw(frame, H, g)
    to_length.fill_(120 + frame)
    start = starts([frame])
    h3.h3_cache_append(to, frame, start, kn, vn, kn.stride(0), kn.stride(1), to_weights)
    o, lse = torch.empty(frame, H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, frame, device="cuda")
    h3.h3_attention_cached(to, h3.make_window(), frame, H, start, qn, qn.stride(0), qn.stride(1), o, lse,
                           ws_of(h3.h3_attention_cached_workspace_bytes(to, frame, H)))
    ok()
    every = np.ones((frame, 120 + frame), bool)
    for h in range(H):
        rows = kept[0, h * Hk // H].long()
        kk = np.concatenate([f64(k[rows, h * Hk // H]), f64(kn[:, h * Hk // H])])
        vv = np.concatenate([f64(v[rows, h * Hk // H]), f64(vn[:, h * Hk // H])])
        (ro, _), (bo, _) = O.forward(f64(qn[:, h]), kk, vv, every)
        within(o.view(frame, H, 128)[:, h], ro, bo, f"after the cut, head {h}")


@pytest.mark.parametrize("lengths, new, H, Hk, page, w", [
    ([1500], [700], 2, 2, 64, dict(right=0)),                                     # six tiles of rows: passes of four and two
    ([1500, 700], [600, 130], 1, 1, 16, dict(left=300, right=0, n_first=200)),    # five and two
    ([900, 64, 513], [385, 1, 300], 6, 2, 128, dict(left=3, right=0, n_first=70, unit=50, origin=70)),
    ([2500, 2100], [129, 2100], 1, 1, 256, dict(left=2, right=1, n_first=0, unit=405, origin=100)),
])
def test_collected_weights_of_many_rows(lengths, new, H, Hk, page, w):
    """Several tiles of rows to a key tile, odd and even many, over one pass and more."""
    test_collected_weights(lengths, new, H, Hk, page, w)


def test_evictions_in_a_row():
    """What the eviction moves early (first, recent, short sequences') is what the call before it left: weights
    collected, then three evictions from pool to pool, none waited for."""
    lengths, heads, page = [3000, 250, 700, 0, 33], 4, 32
    budgets = [(1500, 100, 700), (900, 300, 40), (350, 0, 350)]
    c = Paged(lengths, heads, page, 31)
    stages = [c] + [Paged([min(n, b) for n in lengths], heads, page, 32 + i) for i, (b, _, _) in enumerate(budgets)]
    new = [5, 5, 5, 0, 5]
    start, rows = starts(new), sum(new)
    q = draw(rows, heads, torch.Generator().manual_seed(8))
    lse = torch.full((heads, rows), 3.0, device="cuda")

    def run(wait):
        weights = [torch.full_like(x.w, float("nan")) for x in stages]
        pools = [(c.k, c.v)] + [(torch.full_like(x.k, 3.0), torch.full_like(x.v, 3.0)) for x in stages[1:]]
        lens = [c.length] + [torch.zeros_like(x.length) for x in stages[1:]]
        caches = [h3.make_cache(k, v, x.table, n) for (k, v), x, n in zip(pools, stages, lens)]
        kept = [torch.zeros(len(lengths), heads, b, dtype=torch.int32, device="cuda") for b, _, _ in budgets]
        torch.cuda.synchronize()
        h3.h3_cache_weights(c.cache, h3.make_window(right=0), rows, heads, start, q, q.stride(0), q.stride(1), lse, c.w,
                            weights[0])
        for i, (b, first, recent) in enumerate(budgets):
            if wait:
                torch.cuda.synchronize()
            h3.h3_cache_evict(caches[i], caches[i + 1], b, first, recent, weights[i], weights[i + 1], kept[i], lens[i + 1])
        ok()
        return weights[1:] + [t for pair in pools[1:] for t in pair] + kept + lens[1:]

    slow = run(True)
    assert slow[-1].tolist() == [min(n, 350) for n in lengths]
    for _ in range(5):
        for a, b in zip(run(False), slow):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
