"""Measured cases of the operators for long clips in windows: attention with a sliding window and first keys that
stay visible, its gradient, attention of new rows over a paged cache of keys and values (with the append that
fills it), the attention weight that each cached row collects, and the eviction that goes by it.

listed() and draw() give cases, prepare() makes a case's inputs on the GPU, run() makes one pass (in
elementary torch operations, or with `own` through the library's entry points), exact() gives the same
outputs from the definitions in 64 bits, work() counts what a pass cannot do without.
"""
from __future__ import annotations

import math

import torch

own = False

HEAD = 128                              # channels of an attention head
SCALE = 1.0 / math.sqrt(HEAD)
LARGEST_PAIRS = 15860 ** 2 * 56         # row pairs times heads of the largest listed attention
EXACT_PAIRS = 4_000_000_000             # above this many, 64 bits take too long
AT_ONCE = 1 << 31                       # scores that the plain forms hold at a time


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the tiny block's 72 rows (8 of text, three frames of 16, audio), frames that see themselves, the frame
        # before and the text: launch latency counts
        {"name": "window tiny", "op": "window", "rows": 72, "heads": 4, "kv_heads": 4, "left": 1, "right": 0,
         "first": 8, "unit": 16, "origin": 8, "packed": True},
        # the denoiser's long document with its 405-row frames generated in order: seven frames back and the text
        {"name": "window long", "op": "window", "rows": 15860, "heads": 56, "kv_heads": 56, "left": 7, "right": 0,
         "first": 256, "unit": 405, "origin": 256, "packed": True},
        # a training step of the full-width block over a short clip in frames of 60 rows
        {"name": "window_backward block", "op": "window_backward", "rows": 505, "heads": 56, "kv_heads": 56, "left": 2,
         "right": 0, "first": 17, "unit": 60, "origin": 17, "packed": True},
        # heads that share keys and values, a window to both sides, rows that end inside a tile
        {"name": "window_backward shared", "op": "window_backward", "rows": 4099, "heads": 24, "kv_heads": 4,
         "left": 511, "right": 128, "first": 3, "unit": 1, "origin": 0, "packed": False},
        # a training step over the long document in frames
        {"name": "window_backward long", "op": "window_backward", "rows": 15860, "heads": 56, "kv_heads": 56, "left": 7,
         "right": 0, "first": 256, "unit": 405, "origin": 256, "packed": True},
        # one new row of one document over a cache as long as the whole clip
        {"name": "cached token", "op": "cached", "seqs": 1, "new": 1, "length": 15860, "ragged": False, "heads": 56,
         "kv_heads": 56, "page": 64, "left": -1, "right": 0, "first": 0, "unit": 1, "origin": 0},
        # single rows of a batch of documents of very different lengths, shared keys, small pages
        {"name": "cached batch", "op": "cached", "seqs": 24, "new": 1, "length": 8192, "ragged": True, "heads": 32,
         "kv_heads": 8, "page": 16, "left": -1, "right": 0, "first": 0, "unit": 1, "origin": 0},
        # the next frame of a clip: 405 rows that see themselves, twelve frames back and the text
        {"name": "cached frame", "op": "cached", "seqs": 1, "new": 405, "length": 14836, "ragged": False, "heads": 56,
         "kv_heads": 56, "page": 128, "left": 12, "right": 0, "first": 256, "unit": 405, "origin": 256},
        # what single rows of a batch add to the weights of their cached rows
        {"name": "weights batch", "op": "weights", "seqs": 8, "new": 1, "length": 4096, "ragged": True, "heads": 32,
         "kv_heads": 8, "page": 32, "left": -1, "right": 0, "first": 0, "unit": 1, "origin": 0},
        # what a whole new frame adds, all rows back to the first
        {"name": "weights frame", "op": "weights", "seqs": 1, "new": 405, "length": 14836, "ragged": False, "heads": 56,
         "kv_heads": 56, "page": 128, "left": -1, "right": 0, "first": 0, "unit": 405, "origin": 256},
        # caches of a few documents cut back by an odd number of rows
        {"name": "evict batch", "op": "evict", "seqs": 6, "length": 1111, "ragged": True, "kv_heads": 8, "page": 16,
         "budget": 700, "first": 4, "recent": 64},
        # the long clip's cache cut to half, the text and the last two frames kept
        {"name": "evict long", "op": "evict", "seqs": 1, "length": 15860, "ragged": False, "kv_heads": 56, "page": 128,
         "budget": 7930, "first": 256, "recent": 810},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_heads(rng):
    kv_heads = rng.choice([1, 2, 3, 4, 8, rng.randint(1, 56)])
    shared = rng.choice([1, 1, 2, 4, 7, 8])
    return min(shared, max(1, 56 // kv_heads)) * kv_heads, kv_heads


def _draw_window(rng, rows):
    unit = rng.choice([1, 1, 16, rng.randint(2, 500)])
    span = max(1, rows // unit)
    return {"left": rng.choice([-1, 0, _log_int(rng, 1, span + 1)]),
            "right": rng.choice([0, 0, -1, _log_int(rng, 1, span + 1)]),
            "first": rng.choice([0, 1, 4, rng.randint(0, 300)]), "unit": unit,
            "origin": rng.choice([0, 0, rng.randint(1, 256)])}


def draw(rng):
    op = rng.choice(["window", "window", "window_backward", "window_backward", "cached", "cached", "cached",
                     "weights", "evict"])
    heads, kv_heads = _draw_heads(rng)
    if op.startswith("window"):
        # the gradient from two rows and, with a window of one unit, from whole units on: the softmax over a single
        # key is constant, and its gradient zero
        rows = _log_int(rng, 1 if op == "window" else 2, min(16384, math.isqrt(LARGEST_PAIRS // heads)))
        window = _draw_window(rng, rows)
        if op == "window_backward" and window["left"] == window["right"] == 0:
            window.update(unit=max(window["unit"], 16), origin=0)
        return {"op": op, "rows": rows, "heads": heads, "kv_heads": kv_heads, **window,
                "packed": heads == kv_heads and rng.random() < 0.5}
    page = rng.choice([16, 32, 64, 128, 256])
    seqs = _log_int(rng, 1, 48)
    length = _log_int(rng, 2, max(2, min(32768, 15860 * 56 // (seqs * kv_heads))))
    ragged = seqs > 1 and rng.random() < 0.7
    if op == "evict":
        budget = rng.randint(1, length)
        first = min(budget, rng.choice([0, 4, 64]))
        return {"op": op, "seqs": seqs, "length": length, "ragged": ragged, "kv_heads": kv_heads, "page": page,
                "budget": budget, "first": first, "recent": rng.randint(0, budget - first)}
    most = min(length, 8192, LARGEST_PAIRS // 8 // (seqs * heads * length) + 1)
    new = rng.choice([1, rng.randint(1, min(8, most)), _log_int(rng, 1, most)])
    return {"op": op, "seqs": seqs, "new": new, "length": length, "ragged": ragged, "heads": heads,
            "kv_heads": kv_heads, "page": page, **_draw_window(rng, length)}


def _lengths(case):
    """Cached rows of each document, its new ones among them; ragged: down to about a quarter of the longest."""
    n, length = case["seqs"], case["length"]
    least = case.get("new", 1)
    if not case["ragged"]:
        return [length] * n
    return [max(least, length - 3 * length * s // (4 * n) - (s * s) % 7) for s in range(n)]


def _new_rows(case):
    """New rows of each document; ragged: down to about half of the most."""
    n, new = case["seqs"], case["new"]
    return [new - new * s // (2 * n) if case["ragged"] else new for s in range(n)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _rms_rows(x):
    return x / x.square().mean(-1, keepdim=True).sqrt()


def _normed(rows, heads, g):
    """Queries or keys as the per-head norm leaves them: unit root mean square times learned gains near 1."""
    gain = 1.0 + 0.1 * torch.randn(HEAD, generator=g, device="cuda")
    return (_rms_rows(torch.randn(rows, heads, HEAD, generator=g, device="cuda")) * gain).to(torch.bfloat16)


def _values(rows, heads, g):
    return torch.randn(rows, heads, HEAD, generator=g, device="cuda").to(torch.bfloat16)


def _prepare_window(case, g):
    s, h, hk = case["rows"], case["heads"], case["kv_heads"]
    q, k, v = _normed(s, h, g), _normed(s, hk, g), _values(s, hk, g)
    if case["packed"]:
        qkv = torch.stack([q, k, v], dim=2).contiguous()
        q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    state = {"q": q, "k": k, "v": v}
    if case["op"] == "window_backward":
        state["d_o"] = torch.randn(s, h * HEAD, generator=g, device="cuda").to(torch.bfloat16)
        # what the forward pass leaves: its output and the logarithm of each row's sum
        o, lse = _attend(q, k, v, _visible(case, 0, s, s))
        state["o"], state["lse"] = o.to(torch.bfloat16), lse
    return state


def _pool(case, lengths, g):
    """Pages of a pool, a little larger than needed and handed out in no order, and each document's table."""
    page = case["page"]
    need = [-(-n // page) for n in lengths]
    width, n_pages = max(need), sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return n_pages, table


def _prepare_cache(case, g):
    lengths = _lengths(case)
    n_pages, table = _pool(case, lengths, g)
    rows, hk = n_pages * case["page"], case["kv_heads"]
    shape = (n_pages, case["page"], hk, HEAD)
    paged = lambda t: t.reshape(shape).transpose(1, 2).contiguous()  # noqa: E731
    return {"k_pages": paged(_normed(rows, hk, g)), "v_pages": paged(_values(rows, hk, g)), "table": table,
            "length": torch.tensor(lengths, dtype=torch.int32, device="cuda")}


def _prepare_cached(case, g):
    state = _prepare_cache(case, g)
    new = _new_rows(case)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    rows, h, hk = start[-1], case["heads"], case["kv_heads"]
    state["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    state["q"] = _normed(rows, h, g)
    if case["op"] == "cached":
        state["k"], state["v"] = _normed(rows, hk, g), _values(rows, hk, g)
        return state
    # the rows' own log-sum-exp, as the attention call leaves it, and the weights collected so far
    state["lse"] = _plain_rows(case, state)[1]
    shape = state["k_pages"].shape[:3]
    state["weights"] = torch.empty(shape, device="cuda").exponential_(generator=g)
    return state


def _prepare_evict(case, g):
    state = _prepare_cache(case, g)
    weights = torch.empty(state["k_pages"].shape[:3], device="cuda").exponential_(generator=g)
    # rows that nothing has looked at yet: equal weights
    weights[torch.rand(weights.shape, generator=g, device="cuda") < 0.05] = 0.0
    state["weights"] = weights
    kept = [min(n, case["budget"]) for n in _lengths(case)]
    n_pages, state["to_table"] = _pool(case, kept, g)
    shape = (n_pages,) + tuple(state["k_pages"].shape[1:])
    state["to_k"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    state["to_v"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    state["to_weights"] = torch.zeros(shape[:3], device="cuda")
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = {"window": _prepare_window, "window_backward": _prepare_window, "cached": _prepare_cached,
            "weights": _prepare_cached, "evict": _prepare_evict}[case["op"]]
    return {"case": case, **make(case, g)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"window": _own_window, "window_backward": _own_window_backward, "cached": _own_cached,
                "weights": _own_weights, "evict": _own_evict}[op](state)
    return {"window": _plain_window, "window_backward": _plain_window_backward, "cached": _plain_cached,
            "weights": _plain_weights, "evict": _plain_evict}[op](state)


def _visible(case, at, rows, keys):
    """[rows][keys]: rows stand at positions at, at + 1, ...; a unit is `unit` rows, counted from row `origin`.  A
    row sees the units from `left` before its own to `right` after it (-1: all of them), and of the keys that are
    not after those the first ones."""
    i = torch.arange(at, at + rows, device="cuda").unsqueeze(1)
    j = torch.arange(keys, device="cuda").unsqueeze(0)
    unit_i = torch.div(i - case["origin"], case["unit"], rounding_mode="floor")
    unit_j = torch.div(j - case["origin"], case["unit"], rounding_mode="floor")
    seen = torch.ones(rows, keys, dtype=torch.bool, device="cuda")
    if case["left"] >= 0:
        seen = (unit_j >= unit_i - case["left"]) | (j < case["first"])
    if case["right"] >= 0:
        seen = seen & (unit_j <= unit_i + case["right"])
    return seen


def _attend(q, k, v, visible):
    """softmax(q k^T / sqrt(128)) v over the visible keys, in 32 bits: [rows][heads * 128] and the logarithm of each
    row's sum, [heads][rows]; a row that sees nothing gives zeros and minus infinity."""
    rows, h, keys, hk = q.shape[0], q.shape[1], k.shape[0], k.shape[1]
    shared = h // hk
    qh = q.float().transpose(0, 1).reshape(hk, shared, rows, HEAD)
    kh, vh = k.float().transpose(0, 1).unsqueeze(1), v.float().transpose(0, 1).unsqueeze(1)
    o = torch.empty(hk, shared, rows, HEAD, device="cuda")
    lse = torch.empty(hk, shared, rows, device="cuda")
    step = max(1, AT_ONCE // (shared * rows * max(keys, 1)))
    hidden = ~visible
    for a in range(0, hk, step):
        p = torch.matmul(qh[a:a + step], kh[a:a + step].transpose(2, 3)).mul_(SCALE)
        p.masked_fill_(hidden, -math.inf)
        most = p.amax(-1, keepdim=True)
        most = torch.where(most == -math.inf, torch.zeros_like(most), most)
        p = p.sub_(most).exp_()
        total = p.sum(-1, keepdim=True)
        part = torch.matmul(p, vh[a:a + step]) / total
        o[a:a + step] = torch.where(total > 0, part, torch.zeros_like(part))
        lse[a:a + step] = (most + total.log()).squeeze(-1)
    return o.reshape(h, rows, HEAD).transpose(0, 1).reshape(rows, h * HEAD), lse.reshape(h, rows)


def _plain_window(state):
    s = state["case"]["rows"]
    o, lse = _attend(state["q"], state["k"], state["v"], _visible(state["case"], 0, s, s))
    return {"o": o.to(torch.bfloat16), "lse": lse}


def _plain_window_backward(state):
    """P = exp(q k^T / sqrt(d) - lse) over the visible keys; dV = P^T dO; dS = P (dO V^T - rowsum(dO O)) / sqrt(d);
    dQ = dS K; dK = dS^T Q; dK and dV summed over the heads that share them."""
    case = state["case"]
    s, h, hk = case["rows"], case["heads"], case["kv_heads"]
    shared = h // hk
    by_q = lambda t: t.reshape(s, hk, shared, HEAD).float().permute(1, 2, 0, 3)  # noqa: E731
    q, o, d_o = (by_q(state[n]) for n in ("q", "o", "d_o"))
    k, v = (state[n].float().transpose(0, 1).unsqueeze(1) for n in ("k", "v"))
    lse = state["lse"].reshape(hk, shared, s, 1)
    hidden = ~_visible(case, 0, s, s)
    dq = torch.empty(hk, shared, s, HEAD, device="cuda")
    dk, dv = torch.empty(hk, s, HEAD, device="cuda"), torch.empty(hk, s, HEAD, device="cuda")
    step = max(1, AT_ONCE // (shared * s * s))
    for a in range(0, hk, step):
        b = slice(a, a + step)
        p = torch.matmul(q[b], k[b].transpose(2, 3)).mul_(SCALE).sub_(lse[b]).exp_().masked_fill_(hidden, 0.0)
        dv[b] = torch.matmul(p.transpose(2, 3), d_o[b]).sum(1)
        ds = torch.matmul(d_o[b], v[b].transpose(2, 3)).sub_((d_o[b] * o[b]).sum(-1, keepdim=True)).mul_(p)
        del p
        dq[b] = torch.matmul(ds, k[b]).mul_(SCALE)
        dk[b] = torch.matmul(ds.transpose(2, 3), q[b]).sum(1).mul_(SCALE)
    rows = lambda t: t.to(torch.bfloat16)  # noqa: E731
    return {"dq": rows(dq.reshape(h, s, HEAD).transpose(0, 1)), "dk": rows(dk.transpose(0, 1)),
            "dv": rows(dv.transpose(0, 1))}


def _slots(state, s, first, last):
    """Page and place of a document's slots first .. last - 1."""
    page = state["case"]["page"]
    at = torch.arange(first, last, device="cuda")
    return state["table"][s][torch.div(at, page, rounding_mode="floor")].long(), at % page


def _plain_rows(case, state):
    """Attention of every document's new rows over its cached ones."""
    o = torch.empty(state["q"].shape[0], case["heads"] * HEAD, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(case["heads"], state["q"].shape[0], device="cuda")
    row = 0
    for s, (n, new) in enumerate(zip(_lengths(case), _new_rows(case))):
        where, place = _slots({"case": case, **state}, s, 0, n)
        k, v = state["k_pages"][where, :, place], state["v_pages"][where, :, place]
        part, sums = _attend(state["q"][row:row + new], k, v, _visible(case, n - new, new, n))
        o[row:row + new], lse[:, row:row + new] = part.to(torch.bfloat16), sums
        row += new
    return o, lse


def _plain_cached(state):
    case, row = state["case"], 0
    for s, (n, new) in enumerate(zip(_lengths(case), _new_rows(case))):
        where, place = _slots(state, s, n - new, n)
        state["k_pages"][where, :, place] = state["k"][row:row + new]
        state["v_pages"][where, :, place] = state["v"][row:row + new]
        row += new
    o, lse = _plain_rows(case, state)
    return {"o": o, "lse": lse, "k": state["k_pages"], "v": state["v_pages"]}


def _plain_weights(state):
    """Every cached row's weight plus the sum of its probabilities over the new rows and the heads that share it."""
    case, row = state["case"], 0
    hk, shared = case["kv_heads"], case["heads"] // case["kv_heads"]
    weights = state["weights"].clone()
    for s, (n, new) in enumerate(zip(_lengths(case), _new_rows(case))):
        where, place = _slots(state, s, 0, n)
        k = state["k_pages"][where, :, place].float().permute(1, 2, 0).unsqueeze(1)
        q = state["q"][row:row + new].float().transpose(0, 1).reshape(hk, shared, new, HEAD)
        lse = state["lse"][:, row:row + new].reshape(hk, shared, new, 1)
        hidden = ~_visible(case, n - new, new, n)
        sums = torch.empty(hk, n, device="cuda")
        step = max(1, AT_ONCE // (shared * new * n))
        for a in range(0, hk, step):
            b = slice(a, a + step)
            p = torch.matmul(q[b], k[b]).mul_(SCALE).sub_(lse[b]).exp_().masked_fill_(hidden, 0.0)
            sums[b] = p.sum((1, 2))
        weights[where, :, place] = weights[where, :, place] + sums.transpose(0, 1)
        row += new
    return {"weights": weights}


def _plain_evict(state):
    """Of each document and head the first and the most recent rows and, of the others, those of the largest weight
    (the earlier one of equal ones), in their order, into pages of their own."""
    case = state["case"]
    hk, page, budget = case["kv_heads"], case["page"], case["budget"]
    kept = torch.full((case["seqs"], hk, budget), -1, dtype=torch.int32, device="cuda")
    heads = torch.arange(hk, device="cuda").unsqueeze(1)
    counts = []
    for s, n in enumerate(_lengths(case)):
        where, place = _slots(state, s, 0, n)
        weight = state["weights"][where, :, place].transpose(0, 1)
        many = min(n, budget)
        if n > budget:
            middle = weight[:, case["first"]:n - case["recent"]]
            order = torch.sort(middle, dim=1, descending=True, stable=True).indices + case["first"]
            chosen = order[:, :budget - case["first"] - case["recent"]]
            ends = torch.cat([torch.arange(case["first"], device="cuda"),
                              torch.arange(n - case["recent"], n, device="cuda")]).expand(hk, -1)
            rows = torch.cat([chosen, ends], dim=1).sort(dim=1).values
        else:
            rows = torch.arange(n, device="cuda").expand(hk, -1)
        kept[s, :, :many] = rows.to(torch.int32)
        at = torch.arange(many, device="cuda")
        to_page = state["to_table"][s][torch.div(at, page, rounding_mode="floor")].long().unsqueeze(0)
        for source, target in (("k_pages", "to_k"), ("v_pages", "to_v"), ("weights", "to_weights")):
            state[target][to_page, heads, (at % page).unsqueeze(0)] = state[source][where[rows], heads, place[rows]]
        counts.append(many)
    return {"kept": kept, "length": torch.tensor(counts, dtype=torch.int32, device="cuda"), "k": state["to_k"],
            "v": state["to_v"], "weights": state["to_weights"]}


# ---------------------------------------------------------------------------
# one pass through the library; buffers, workspace and configuration are kept with the state, as a program
# that calls the operator every step keeps them
# ---------------------------------------------------------------------------

def _window_of(case):
    import audio_video_flow_gb300 as h3
    return h3.make_window(case["left"], case["right"], case["first"], case["unit"], case["origin"])


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def _own_window(state):
    import audio_video_flow_gb300 as h3
    case, q, k = state["case"], state["q"], state["k"]
    s, h, hk = case["rows"], case["heads"], case["kv_heads"]
    kept = state.get("own")
    if kept is None:
        out = {"o": torch.empty(s, h * HEAD, dtype=torch.bfloat16, device="cuda"),
               "lse": torch.empty(h, s, device="cuda")}
        kept = state["own"] = _window_of(case), out, _bytes(h3.h3_attention_window_workspace_bytes(s, h, hk))
    window, out, ws = kept
    h3.h3_attention_window(window, s, h, hk, q, q.stride(0), q.stride(1), k, state["v"], k.stride(0), k.stride(1),
                           out["o"], out["lse"], ws)
    return out


def _own_window_backward(state):
    import audio_video_flow_gb300 as h3
    case, q, k = state["case"], state["q"], state["k"]
    s, h, hk = case["rows"], case["heads"], case["kv_heads"]
    kept = state.get("own")
    if kept is None:
        rows = lambda n: torch.empty(s, n, HEAD, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        out = {"dq": rows(h), "dk": rows(hk), "dv": rows(hk)}
        kept = state["own"] = _window_of(case), out, _bytes(h3.h3_attention_window_backward_workspace_bytes(s, h, hk))
    window, out, ws = kept
    h3.h3_attention_window_backward(window, s, h, hk, q, q.stride(0), q.stride(1), k, state["v"], k.stride(0),
                                    k.stride(1), state["o"], state["d_o"], state["lse"], out["dq"], h * HEAD, HEAD,
                                    out["dk"], out["dv"], hk * HEAD, HEAD, ws)
    return out


def _own_cache(state):
    import audio_video_flow_gb300 as h3
    return h3.make_cache(state["k_pages"], state["v_pages"], state["table"], state["length"])


def _own_cached(state):
    import audio_video_flow_gb300 as h3
    case, q, k = state["case"], state["q"], state["k"]
    rows, h = q.shape[0], case["heads"]
    kept = state.get("own")
    if kept is None:
        cache = _own_cache(state)
        out = {"o": torch.empty(rows, h * HEAD, dtype=torch.bfloat16, device="cuda"),
               "lse": torch.empty(h, rows, device="cuda"), "k": state["k_pages"], "v": state["v_pages"]}
        kept = state["own"] = cache, _window_of(case), out, _bytes(h3.h3_attention_cached_workspace_bytes(cache, rows, h))
    cache, window, out, ws = kept
    h3.h3_cache_append(cache, rows, state["start"], k, state["v"], k.stride(0), k.stride(1))
    h3.h3_attention_cached(cache, window, rows, h, state["start"], q, q.stride(0), q.stride(1), out["o"], out["lse"], ws)
    return out


def _own_weights(state):
    import audio_video_flow_gb300 as h3
    case, q = state["case"], state["q"]
    kept = state.get("own")
    if kept is None:
        # pages of no document keep what they hold
        kept = state["own"] = _own_cache(state), _window_of(case), state["weights"].clone()
    cache, window, out = kept
    h3.h3_cache_weights(cache, window, q.shape[0], case["heads"], state["start"], q, q.stride(0), q.stride(1),
                        state["lse"], state["weights"], out)
    return {"weights": out}


def _own_evict(state):
    import audio_video_flow_gb300 as h3
    case = state["case"]
    kept = state.get("own")
    if kept is None:
        length = torch.empty(case["seqs"], dtype=torch.int32, device="cuda")
        out = {"kept": torch.empty(case["seqs"], case["kv_heads"], case["budget"], dtype=torch.int32, device="cuda"),
               "length": length, "k": state["to_k"], "v": state["to_v"], "weights": state["to_weights"]}
        to = h3.make_cache(state["to_k"], state["to_v"], state["to_table"], length)
        kept = state["own"] = _own_cache(state), to, out
    cache, to, out = kept
    h3.h3_cache_evict(cache, to, case["budget"], case["first"], case["recent"], state["weights"], out["weights"],
                      out["kept"], out["length"])
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_bounds(case, at, rows, keys):
    """First and last + 1 of each row's window, from the units' borders."""
    lo, hi = [], []
    for i in range(at, at + rows):
        unit = (i - case["origin"]) // case["unit"]
        lo.append(0 if case["left"] < 0 else case["origin"] + (unit - case["left"]) * case["unit"])
        hi.append(keys if case["right"] < 0 else case["origin"] + (unit + case["right"] + 1) * case["unit"])
    return (torch.tensor(t, device="cuda").clamp(0, keys).unsqueeze(1) for t in (lo, hi))


def _exact_scores(case, q, k, at):
    """[kv_heads][shared][rows][keys] scores, minus infinity where a row does not see the key."""
    rows, keys, hk = q.shape[0], k.shape[0], k.shape[1]
    s = torch.einsum("ihgc,jhc->hgij", q.double().reshape(rows, hk, -1, HEAD), k.double()) / math.sqrt(HEAD)
    lo, hi = _exact_bounds(case, at, rows, keys)
    j = torch.arange(keys, device="cuda")
    return torch.where((j < hi) & ((j >= lo) | (j < case["first"])), s, torch.full_like(s, -math.inf))


def _exact_attention(case, q, k, v, at):
    s = _exact_scores(case, q, k, at)
    lse = torch.logsumexp(s, -1)
    o = torch.einsum("hgij,jhc->ihgc", torch.exp(s - lse.unsqueeze(-1)), v.double())
    return o.reshape(q.shape[0], -1), lse.reshape(-1, q.shape[0])


def exact(case, seed):
    op = case["op"]
    if op.startswith("window"):
        pairs = case["rows"] ** 2 * case["heads"]
    elif op == "evict":
        pairs = 0
    else:
        pairs = sum(n * new for n, new in zip(_lengths(case), _new_rows(case))) * case["heads"]
    if pairs > EXACT_PAIRS:
        return None
    st = prepare(case, seed)
    if op == "window":
        o, lse = _exact_attention(case, st["q"], st["k"], st["v"], 0)
        return {"o": o, "lse": lse}
    if op == "window_backward":
        n, hk = case["rows"], case["kv_heads"]
        q, k, v = st["q"].double().reshape(n, hk, -1, HEAD), st["k"].double(), st["v"].double()
        o, d_o = (st[name].double().reshape(n, hk, -1, HEAD) for name in ("o", "d_o"))
        p = torch.exp(_exact_scores(case, st["q"], st["k"], 0) - st["lse"].double().reshape(hk, -1, n, 1))
        dv = torch.einsum("hgij,ihgc->jhc", p, d_o)
        delta = torch.einsum("ihgc,ihgc->hgi", d_o, o)
        p *= torch.einsum("ihgc,jhc->hgij", d_o, v) - delta.unsqueeze(-1)
        p /= math.sqrt(HEAD)
        return {"dq": torch.einsum("hgij,jhc->ihgc", p, k).reshape(n, -1, HEAD),
                "dk": torch.einsum("hgij,ihgc->jhc", p, q), "dv": dv}
    table, page, row = st["table"].tolist(), case["page"], 0
    if op == "evict":
        return _exact_evict(case, st, table)
    flat = {name: st[name].transpose(1, 2).reshape(-1, case["kv_heads"], HEAD).clone() for name in ("k_pages", "v_pages")}
    o, lses = [], []
    weights = st["weights"].double().transpose(1, 2).reshape(-1, case["kv_heads"]) if op == "weights" else None
    for s, (n, new) in enumerate(zip(_lengths(case), _new_rows(case))):
        slots = torch.tensor([table[s][i // page] * page + i % page for i in range(n)], device="cuda")
        q = st["q"][row:row + new]
        if op == "weights":
            score = _exact_scores(case, q, flat["k_pages"][slots], n - new)
            lse = st["lse"][:, row:row + new].double().reshape(case["kv_heads"], -1, new, 1)
            weights[slots] += torch.exp(score - lse).sum((1, 2)).transpose(0, 1)
        else:
            flat["k_pages"][slots[n - new:]] = st["k"][row:row + new]
            flat["v_pages"][slots[n - new:]] = st["v"][row:row + new]
            part, lse = _exact_attention(case, q, flat["k_pages"][slots], flat["v_pages"][slots], n - new)
            o.append(part)
            lses.append(lse)
        row += new
    if op == "weights":
        return {"weights": weights.reshape(-1, page, case["kv_heads"]).transpose(1, 2)}
    pages = {name: flat[name].reshape(-1, page, case["kv_heads"], HEAD).transpose(1, 2) for name in flat}
    return {"o": torch.cat(o), "lse": torch.cat(lses, dim=1), "k": pages["k_pages"], "v": pages["v_pages"]}


def _exact_evict(case, st, table):
    import numpy as np
    page, hk, budget = case["page"], case["kv_heads"], case["budget"]
    weights = st["weights"].cpu().numpy()
    kept = np.full((case["seqs"], hk, budget), -1, np.int32)
    lengths = _lengths(case)
    out = {name: torch.zeros_like(st[to]) for name, to in (("k", "to_k"), ("v", "to_v"), ("weights", "to_weights"))}
    to_table = st["to_table"].tolist()
    for s, n in enumerate(lengths):
        where = np.array([table[s][i // page] for i in range(n)])
        place = np.arange(n) % page
        many = min(n, budget)
        target = torch.tensor([to_table[s][i // page] for i in range(many)], device="cuda")
        for h in range(hk):
            rank = np.zeros(n, np.int64)   # 0: kept whatever its weight
            if n > budget:
                free = np.arange(case["first"], n - case["recent"])
                order = free[np.lexsort((free, -weights[where[free], h, place[free]].astype(np.float64)))]
                rank[order] = np.arange(1, len(order) + 1)
            rows = np.nonzero(rank <= budget - case["first"] - case["recent"])[0] if n > budget else np.arange(n)
            kept[s, h, :many] = rows
            source = torch.from_numpy(where[rows]).cuda(), torch.from_numpy(place[rows]).cuda()
            at = torch.arange(many, device="cuda") % page
            for name, pages in (("k", "k_pages"), ("v", "v_pages"), ("weights", "weights")):
                out[name][target, h, at] = st[pages][source[0], h, source[1]]
    return {"kept": torch.from_numpy(kept), "length": torch.tensor([min(n, budget) for n in lengths], dtype=torch.int32),
            **out}


# ---------------------------------------------------------------------------
# work of one pass
# ---------------------------------------------------------------------------

def _seen(case, at, rows, keys):
    """Visible pairs of row and key, and the keys that some row sees."""
    pairs, seen_lo, seen_hi, to_first = 0, keys, 0, 0
    unit, origin, first = case["unit"], case["origin"], case["first"]
    i, last = at, at + rows
    while i < last:   # the rows of one unit see the same keys
        u = (i - origin) // unit
        n = min(last, origin + (u + 1) * unit) - i
        lo = 0 if case["left"] < 0 else min(keys, max(0, origin + (u - case["left"]) * unit))
        hi = keys if case["right"] < 0 else min(keys, max(0, origin + (u + case["right"] + 1) * unit))
        extra = min(first, lo, hi)
        pairs += n * (max(0, hi - lo) + extra)
        if hi > lo:
            seen_lo, seen_hi = min(seen_lo, lo), max(seen_hi, hi)
        to_first = max(to_first, extra)
        i += n
    return pairs, max(0, seen_hi - seen_lo) + min(to_first, seen_lo)


def work(case):
    op, hk = case["op"], case["kv_heads"]
    row = HEAD * 2
    if op.startswith("window"):
        s, h = case["rows"], case["heads"]
        pairs = _seen(case, 0, s, s)[0]
        if op == "window":
            # reads q, k and v, writes o and lse; two products
            return {"bytes": s * (2 * h * row + 2 * hk * row + 4 * h), "flops": 4 * pairs * h * HEAD}
        # reads q, k, v, o, dO and lse, writes dq, dk and dv; five products
        return {"bytes": s * (4 * h * row + 4 * hk * row + 4 * h), "flops": 10 * pairs * h * HEAD}
    lengths = _lengths(case)
    if op == "evict":
        kept = sum(min(n, case["budget"]) for n in lengths)
        # reads every weight, reads and writes the kept rows, their weights and places
        return {"bytes": hk * (4 * sum(lengths) + kept * (4 * row + 3 * 4)), "flops": hk * sum(lengths)}
    h, pairs, keys, new = case["heads"], 0, 0, sum(_new_rows(case))
    for n, more in zip(lengths, _new_rows(case)):
        p, seen = _seen(case, n - more, more, n)
        pairs += p
        keys += seen
    if op == "weights":
        # reads q, lse, the visible keys and every weight, writes the weights; one product
        return {"bytes": new * h * (row + 4) + hk * (keys * row + sum(lengths) * 8), "flops": 2 * pairs * h * HEAD}
    # reads q, the new k and v and the visible cached ones, writes the new ones, o and lse; two products
    return {"bytes": new * (2 * h * row + 4 * h + 4 * hk * row) + max(0, keys - new) * hk * 2 * row,
            "flops": 4 * pairs * h * HEAD}
