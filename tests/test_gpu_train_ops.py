"""The training-side operators on the GPU against the fp64 oracle: the gradient
of the attention core, rotary positions and their gradient, the row norms and
theirs.  Every comparison is elementwise against the oracle's error bound for
that element (oracle/h3_train_oracle.py derives the bounds from the roundings
each operator makes); nothing is fitted to the results."""
import numpy as np
import pytest
import torch

import audio_video_flow_gb300 as h3
from oracle import h3_train_oracle as O

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": (torch.bfloat16, h3.H3_BF16, O.HALF_BF16), "fp32": (torch.float32, h3.H3_FP32, O.U32)}
KINDS = {"rms": h3.H3_NORM_RMS, "layer": h3.H3_NORM_LAYER}


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def within(got, ref, bound, what):
    got = f64(got) if torch.is_tensor(got) else got
    e = np.abs(got - ref)
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = float((e / np.maximum(bound, 1e-45)).max()) if e.size else 0.0
    assert (e <= bound).all(), f"{what}: error {worst:.3g} times its bound"


def ok():
    torch.cuda.synchronize()
    assert h3.h3_sync_check(timeout_ms=60000) == 0


# ---------------------------------------------------------------------------
# attention backward
# ---------------------------------------------------------------------------

def attention_case(S, H, seed, packed=True, gap=0, std=1.0):
    """q, k, v views, o, d_o, lse on the GPU; o and lse from the oracle's
    forward, as rounded inputs."""
    g = torch.Generator().manual_seed(seed)
    draw = lambda s: (s * torch.randn(S, H, 128, generator=g)).to(torch.bfloat16)  # noqa: E731
    q, k, v, d_o = draw(std), draw(std), draw(1.0), draw(1.0)
    o = torch.empty(S, H, 128, dtype=torch.bfloat16)
    lse = torch.empty(H, S)
    for h in range(H):
        oo, ll = O.attention_forward(f64(q[:, h]), f64(k[:, h]), f64(v[:, h]))
        o[:, h] = torch.from_numpy(oo).to(torch.bfloat16)
        lse[h] = torch.from_numpy(ll).float()
    if packed:
        qkv = torch.stack([q, k, v], dim=2).cuda()
        q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    else:
        wide = lambda t: torch.cat([t, torch.full((S, H, gap), float("nan"), dtype=torch.bfloat16)], 2).cuda()[..., :128]  # noqa: E731
        q, k, v = wide(q), wide(k), wide(v)
    return q, k, v, o.cuda(), d_o.cuda(), lse.cuda()


def attention_backward(case, packed=True, gap=0, stream=None, ws=None, fill=7.0):
    q, k, v, o, d_o, lse = case
    S, H, _ = q.shape
    if packed:
        buf = torch.full((S, H, 3, 128), fill, dtype=torch.bfloat16, device="cuda")
        grads = [buf[:, :, i] for i in range(3)]
    else:
        buf = torch.full((3, S, H, 128 + gap), fill, dtype=torch.bfloat16, device="cuda")
        grads = [buf[i][..., :128] for i in range(3)]
    if ws is None:
        ws = torch.empty(h3.h3_attention_backward_workspace_bytes(S, H), dtype=torch.uint8, device="cuda")
    h3.h3_attention_backward(S, H, q, k, v, q.stride(0), q.stride(1), o, d_o, lse, *grads, grads[0].stride(0),
                             grads[0].stride(1), ws, stream)
    return grads, buf


def check_attention(case, grads, what):
    q, k, v, o, d_o, lse = (f64(t) for t in case)
    for h in range(q.shape[1]):
        ref, bound = O.attention_backward(q[:, h], k[:, h], v[:, h], o[:, h], d_o[:, h], lse[h])
        for name, got in zip(("dq", "dk", "dv"), grads):
            within(f64(got[:, h]), ref[name], bound[name], f"{what} head {h} {name}")


@pytest.mark.parametrize("S", [1, 2, 7, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 505])
def test_attention_backward_lengths(S):
    case = attention_case(S, 2, S)
    grads, _ = attention_backward(case)
    ok()
    check_attention(case, grads, f"S={S}")


@pytest.mark.parametrize("S, H, gap", [(72, 4, 0), (131, 3, 8), (300, 1, 40), (130, 56, 0)])
def test_attention_backward_separate_tensors(S, H, gap):
    case = attention_case(S, H, S + H, packed=False, gap=gap)
    grads, buf = attention_backward(case, packed=False, gap=gap)
    ok()
    check_attention(case, grads, f"S={S} H={H}")
    if gap:
        assert (buf[..., 128:] == 7.0).all()      # what lies between the rows is left as it was


@pytest.mark.parametrize("S", [1, 72, 128, 200, 256])
def test_attention_backward_few_and_many_heads_agree(S):
    """A head's gradient is the same bits whatever heads lie beside it: few
    heads of a short document compute their row values inside the main kernel,
    many take them from the kernel before it."""
    H = 160
    case = attention_case(S, H, S + 17)
    many, _ = attention_backward(case)
    ok()
    for h in (0, 3, 77, H - 2):
        part = tuple(t[:, h:h + 2].contiguous() for t in case[:5]) + (case[5][h:h + 2].contiguous(),)
        few, _ = attention_backward(part)
        ok()
        for name, x, y in zip(("dq", "dk", "dv"), few, many):
            assert torch.equal(x, y[:, h:h + 2]), f"S={S} head {h} {name}"
        if h == 77:
            check_attention(part, few, f"S={S}")


def test_attention_backward_long():
    case = attention_case(4099, 1, 5)
    grads, _ = attention_backward(case)
    ok()
    check_attention(case, grads, "S=4099")


@pytest.mark.parametrize("std", [0.0, 3.0, 8.0])
def test_attention_backward_flat_and_peaked_rows(std):
    """std 0: equal scores; 8: rows that one key decides."""
    case = attention_case(257, 2, 31, std=std)
    grads, _ = attention_backward(case)
    ok()
    check_attention(case, grads, f"std={std}")


@pytest.mark.parametrize("sign", [1, -1])
def test_attention_backward_far_scores(sign):
    """Scores near +-1800 in every row, and rows that end inside a tile: the
    keys past the end must not bring exp(-lse) = inf into dq."""
    S, H = 130, 2
    g = torch.Generator().manual_seed(3)
    u = torch.randn(128, generator=g)
    near = lambda a: (a * u + 0.05 * torch.randn(S, H, 128, generator=g)).to(torch.bfloat16)  # noqa: E731
    q, k = near(12.0), near(12.0 * sign)
    v, d_o = (torch.randn(S, H, 128, generator=g).to(torch.bfloat16) for _ in range(2))
    o, lse = torch.empty(S, H, 128, dtype=torch.bfloat16), torch.empty(H, S)
    for h in range(H):
        oo, ll = O.attention_forward(f64(q[:, h]), f64(k[:, h]), f64(v[:, h]))
        o[:, h], lse[h] = torch.from_numpy(oo).to(torch.bfloat16), torch.from_numpy(ll).float()
    assert (lse.abs() > 1000).all()
    case = tuple(t.cuda() for t in (q, k, v, o, d_o, lse))
    grads, _ = attention_backward(case, packed=False)
    ok()
    check_attention(case, grads, f"far {sign}")


def test_attention_backward_reads_the_forward_calls_outputs():
    """o and lse from h3_attention itself, packed q, k, v."""
    S, H = 333, 3
    q, k, v, o, d_o, lse = attention_case(S, H, 8)
    h3.h3_attention(S, H, q, k, v, q.stride(0), q.stride(1), o, lse)
    case = (q, k, v, o, d_o, lse)
    grads, _ = attention_backward(case)
    ok()
    check_attention(case, grads, "forward's outputs")


def test_attention_backward_repeats_bitwise_and_leaves_inputs():
    case = attention_case(389, 5, 17)
    before = [t.clone() for t in case]
    a, _ = attention_backward(case, fill=7.0)
    b, _ = attention_backward(case, fill=-3.0)
    ok()
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    for x, y in zip(before, case):
        assert torch.equal(x, y)


def test_attention_backward_two_streams_and_graph():
    """Calls on two streams at once, each with its own workspace, and a
    captured call replayed with new contents in its buffers."""
    cases = [attention_case(S, 4, S) for S in (200, 321)]
    alone = [attention_backward(c)[0] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        both = [attention_backward(c, stream=s)[0] for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    # graph: capture on case 0's buffers, then copy other inputs into them
    other = attention_case(200, 4, 99)
    want, _ = attention_backward(other)
    static = [t.clone() for t in cases[0]]
    base = torch.stack([static[0], static[1], static[2]], 2)
    static[:3] = [base[:, :, i] for i in range(3)]
    ws = torch.empty(h3.h3_attention_backward_workspace_bytes(200, 4), dtype=torch.uint8, device="cuda")
    grads = torch.empty(200, 4, 3, 128, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = static[0]
        h3.h3_attention_backward(200, 4, *static[:3], q.stride(0), q.stride(1), *static[3:], grads[:, :, 0],
                                 grads[:, :, 1], grads[:, :, 2], grads.stride(0), grads.stride(1), ws)
    for to, src in zip(static, other):
        to.copy_(src)
    graph.replay()
    graph.replay()
    ok()
    for i in range(3):
        assert torch.equal(grads[:, :, i], want[i])


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

def rope_rows(S, H, width, dtype, seed, gap=0):
    g = torch.Generator().manual_seed(seed)
    unit = 16 // dtype.itemsize
    full = torch.full((S, H, (width + unit - 1) // unit * unit + gap), float("nan"), dtype=dtype)
    full[..., :width] = torch.randn(S, H, width, generator=g).to(dtype)
    return full.cuda()


ROPES = [  # width, axes, freqs
    (128, 3, 16), (128, 1, 64), (128, 1, 32), (64, 1, 32), (80, 1, 20), (96, 2, 12), (256, 1, 128), (40, 3, 5),
    (26, 1, 13), (2, 1, 1), (10, 1, 3), (256, 4, 1), (100, 1, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("width, axes, freqs", ROPES)
def test_rope(width, axes, freqs, layout, dtype):
    tdtype, code, half = DTYPES[dtype]
    S, HQ, HK = 37, 5, 2
    q, k = rope_rows(S, HQ, width, tdtype, 1, gap=8), rope_rows(S, HK, width, tdtype, 2, gap=8)
    both = torch.cat([q, k], 1)
    q, k = both[:, :HQ], both[:, HQ:]
    pos = torch.randint(0, 2000, (S, axes), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    cfg = h3.make_rope_config(width, axes, freqs, dtype=code,
                              layout=h3.H3_ROPE_HALF if layout == "half" else h3.H3_ROPE_INTERLEAVED)
    table = O.rope_frequencies(axes, freqs)
    for direction in (h3.H3_ROPE_FORWARD, h3.H3_ROPE_BACKWARD):
        out = torch.full_like(both, 5.0)
        h3.h3_rope(cfg, S, pos.cuda(), direction, q, out, HQ, k, out[:, HQ:], HK, both.stride(0), both.stride(1),
                   out.stride(0), out.stride(1))
        ok()
        ref, bound = O.rope(f64(both[..., :width]), pos.numpy(), table, layout, backward=direction == h3.H3_ROPE_BACKWARD,
                            half=half)
        within(out[..., :width], ref, bound, f"{layout} {dtype} {direction}")
        assert (out[..., width:] == 5.0).all()
        place = both.clone()                              # in place: the same bits
        h3.h3_rope(cfg, S, pos.cuda(), direction, place, place, HQ, place[:, HQ:], place[:, HQ:], HK, place.stride(0),
                   place.stride(1), place.stride(0), place.stride(1))
        ok()
        assert torch.equal(place[..., :width], out[..., :width])
        assert place[..., width:].isnan().all()


@pytest.mark.parametrize("S, HQ, HK", [(1, 1, 0), (1, 32, 8), (1, 56, 56), (2, 3, 1), (700, 56, 56), (5, 300, 0)])
def test_rope_row_and_head_counts(S, HQ, HK):
    x = rope_rows(S, HQ + HK, 128, torch.bfloat16, 4)
    pos = torch.randint(0, 100, (S, 3), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    cfg = h3.make_rope_config(128, 3, 16)
    out = torch.empty_like(x)
    h3.h3_rope(cfg, S, pos.cuda(), 0, x, out, HQ, x[:, HQ:] if HK else None, out[:, HQ:] if HK else None, HK,
               x.stride(0), x.stride(1), out.stride(0), out.stride(1))
    ok()
    ref, bound = O.rope(f64(x[:, :HQ + HK]), pos.numpy(), O.rope_frequencies(3, 16))
    within(out[:, :HQ + HK], ref, bound, "counts")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("width, axes, freqs", [(128, 3, 16), (64, 1, 32), (26, 1, 13), (100, 1, 16)])
@pytest.mark.parametrize("S, HQ, HK", [(5003, 1, 0), (3331, 2, 1), (9001, 1, 1)])
def test_rope_many_rows_of_few_heads(S, HQ, HK, width, axes, freqs, layout):
    """Several rows to a CTA, the last CTA's not all there."""
    x = rope_rows(S, HQ + HK, width, torch.bfloat16, 4)
    pos = torch.randint(0, 4000, (S, axes), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    cfg = h3.make_rope_config(width, axes, freqs,
                              layout=h3.H3_ROPE_HALF if layout == "half" else h3.H3_ROPE_INTERLEAVED)
    out = torch.full((S + 7, *x.shape[1:]), 5.0, dtype=x.dtype, device="cuda")
    h3.h3_rope(cfg, S, pos.cuda(), 0, x, out, HQ, x[:, HQ:] if HK else None, out[:, HQ:] if HK else None, HK,
               x.stride(0), x.stride(1), out.stride(0), out.stride(1))
    ok()
    ref, bound = O.rope(f64(x[..., :width]), pos.numpy(), O.rope_frequencies(axes, freqs), layout)
    within(out[:S, :, :width], ref, bound, "many rows")
    assert (out[S:] == 5.0).all()


def test_operators_on_head_major_tensors():
    """[heads][rows][128] tensors: the row stride is the smaller one."""
    S, H = 150, 3
    q, k, v, o, d_o, lse = attention_case(S, H, 41)
    major = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
    want, _ = attention_backward((q, k, v, o, d_o, lse))
    grads = [torch.full((H, S, 128), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1) for _ in range(3)]
    ws = torch.empty(h3.h3_attention_backward_workspace_bytes(S, H), dtype=torch.uint8, device="cuda")
    h3.h3_attention_backward(S, H, *major, 128, S * 128, o, d_o, lse, *grads, 128, S * 128, ws)
    ok()
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    pos = torch.randint(0, 99, (S, 1), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    rope, norm = h3.make_rope_config(128, 1, 64), h3.make_norm_config(h3.H3_NORM_LAYER, 128)
    for x in (q.contiguous(), major[0]):
        st = (x.stride(0), x.stride(1))
        y, z, dx = (torch.empty_like(x) for _ in range(3))
        assert y.stride() == x.stride()
        dg, db = (torch.empty(128, device="cuda") for _ in range(2))
        ws = torch.empty(h3.h3_norm_backward_workspace_bytes(norm, S, H), dtype=torch.uint8, device="cuda")
        h3.h3_rope(rope, S, pos, 0, x, y, H, None, None, 0, *st, *st)
        h3.h3_norm_forward(norm, S, H, x, *st, None, None, z, *st)
        h3.h3_norm_backward(norm, S, H, x, *st, None, y, *st, dx, *st, dg, db, ws)
        got = [t.contiguous() for t in (y, z, dx, dg, db)]
        if x is major[0]:
            assert all(torch.equal(a, b) for a, b in zip(got, first))
        first = got
    ok()


def test_operators_on_rows_far_apart():
    """Rows 2^30 elements apart: offsets past 32 bits, in elements and bytes,
    against the same call on packed rows."""
    S, H, far = 5, 2, 1 << 30
    buf = torch.empty((S - 1) * far + 4096, dtype=torch.bfloat16, device="cuda")

    def spread(i, fill=None):      # the i-th [S][H][128] view into buf
        t = buf.as_strided((S, H, 128), (far, 128, 1), 256 * i)
        t.copy_(torch.full_like(t, 7.0) if fill is None else fill)
        return t

    q, k, v, o, d_o, lse = attention_case(S, H, 11, packed=False)
    want, _ = attention_backward((q, k, v, o, d_o, lse), packed=False)
    grads = [spread(3 + i) for i in range(3)]
    ws = torch.empty(h3.h3_attention_backward_workspace_bytes(S, H), dtype=torch.uint8, device="cuda")
    h3.h3_attention_backward(S, H, spread(0, q), spread(1, k), spread(2, v), far, 128, o, d_o, lse, *grads, far, 128,
                             ws)
    ok()
    assert all(torch.equal(a, b) for a, b in zip(grads, want))

    pos = torch.tensor([[0], [1], [2], [77], [1000]], dtype=torch.int32, device="cuda")
    rope, norm = h3.make_rope_config(128, 1, 64), h3.make_norm_config(h3.H3_NORM_LAYER, 128)
    got = []
    for x, dy, y, z, dx, row in [(q, k, *(torch.empty_like(q) for _ in range(3)), H * 128),
                                 (spread(0, q), spread(1, k), *(spread(6 + i) for i in range(3)), far)]:
        dg, db = (torch.empty(128, device="cuda") for _ in range(2))
        ws = torch.empty(h3.h3_norm_backward_workspace_bytes(norm, S, H), dtype=torch.uint8, device="cuda")
        h3.h3_rope(rope, S, pos, 0, x, y, H, None, None, 0, row, 128, row, 128)
        h3.h3_norm_forward(norm, S, H, x, row, 128, None, None, z, row, 128)
        h3.h3_norm_backward(norm, S, H, x, row, 128, None, dy, row, 128, dx, row, 128, dg, db, ws)
        ok()
        got.append((y, z, dx, dg, db))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_rows_past_the_last_are_left():
    """Outputs larger than the call's rows keep what lies behind them."""
    S, H = 70, 2
    case = attention_case(S, H, 6)
    buf = torch.full((S + 80, H, 3, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((h3.h3_attention_backward_workspace_bytes(S, H) + 64,), 9, dtype=torch.uint8, device="cuda")
    q, k, v, o, d_o, lse = case
    h3.h3_attention_backward(S, H, q, k, v, q.stride(0), q.stride(1), o, d_o, lse, buf[:, :, 0], buf[:, :, 1],
                             buf[:, :, 2], buf.stride(0), buf.stride(1), ws[:-64])
    x, dy = norm_rows(S, 1, 300, torch.bfloat16, 1), norm_rows(S, 1, 300, torch.bfloat16, 2)
    y, dx = (torch.full((S + 40, 1, 304), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dg, db = (torch.full((308,), 3.0, device="cuda") for _ in range(2))
    cfg = h3.make_norm_config(h3.H3_NORM_LAYER, 300)
    nws = h3.h3_norm_backward_workspace_bytes(cfg, S, 1)
    ws2 = torch.full((nws + 64,), 9, dtype=torch.uint8, device="cuda")
    h3.h3_norm_forward(cfg, S, 1, x, 304, 304, None, None, y, 304, 304)
    h3.h3_norm_backward(cfg, S, 1, x, 304, 304, None, dy, 304, 304, dx, 304, 304, dg, db, ws2[:nws])
    ok()
    assert (buf[S:] == 7.0).all() and (ws[-64:] == 9).all() and (ws2[nws:] == 9).all()
    assert (y[S:] == 5.0).all() and (dx[S:] == 5.0).all() and (y[:, :, 300:] == 5.0).all()
    assert (dg[300:] == 3.0).all() and (db[300:] == 3.0).all()


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn"])
@pytest.mark.parametrize("scaled_axes", [1, 2, 3])
def test_rope_scalings(scaling, scaled_axes):
    S, H = 64, 3
    x = rope_rows(S, H, 128, torch.float32, 4)
    pos = torch.randint(0, 1 << 17, (S, 2), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    kw = dict(factor=8.0, scaled_axes=scaled_axes, trained_length=4096.0, alpha=1.0, beta=32.0, theta=500000.0)
    codes = {"linear": h3.H3_ROPE_SCALE_LINEAR, "ntk": h3.H3_ROPE_SCALE_NTK, "yarn": h3.H3_ROPE_SCALE_YARN}
    cfg = h3.make_rope_config(128, 2, 32, dtype=h3.H3_FP32, scaling=codes[scaling], magnitude=1.25, **kw)
    out = torch.empty_like(x)
    h3.h3_rope(cfg, S, pos.cuda(), 0, x, out, H, None, None, 0, x.stride(0), x.stride(1), out.stride(0), out.stride(1))
    ok()
    ref, bound = O.rope(f64(x), pos.numpy(), O.rope_frequencies(2, 32, scaling=scaling, **kw), magnitude=1.25, half=O.U32)
    within(out, ref, bound, scaling)


def test_rope_far_and_negative_positions():
    pos = torch.tensor([0, 1, -1, 1 << 20, (1 << 24) + 1, -(1 << 24) - 3, 2 ** 31 - 1, -2 ** 31, 123456789],
                       dtype=torch.int32)[:, None]
    S, H = len(pos), 2
    x = rope_rows(S, H, 128, torch.float32, 4)
    cfg = h3.make_rope_config(128, 1, 64, dtype=h3.H3_FP32)
    out = torch.empty_like(x)
    h3.h3_rope(cfg, S, pos.cuda(), 0, x, out, H, None, None, 0, x.stride(0), x.stride(1), out.stride(0), out.stride(1))
    ok()
    ref, bound = O.rope(f64(x), pos.numpy(), O.rope_frequencies(1, 64), half=O.U32)
    within(out, ref, bound, "far")


def test_rope_matches_the_blocks_own_rotation():
    """h3_rope_qknorm is h3_norm_forward per head followed by h3_rope: each of
    the two rounds to bf16 at the same places, so they differ by the angles'
    fp32 product alone (positions below 64: an error below 2^-17)."""
    S, H = 129, 4
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(S, H, 3, 128, generator=g).to(torch.bfloat16).cuda()
    gains = [(1 + 0.1 * torch.randn(128, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]
    pos = torch.randint(0, 64, (S, 3), generator=g, dtype=torch.int32).cuda()
    mine = qkv.clone()
    cfg = h3.make_config(512, H, 1536, 256)
    h3.h3_rope_qknorm(cfg, S, pos, qkv[:, :, 0], qkv[:, :, 1], H * 384, 384, *gains)
    norm, rope = h3.make_norm_config(h3.H3_NORM_RMS, 128), h3.make_rope_config(128, 3, 16)
    for i in range(2):
        t = mine[:, :, i]
        h3.h3_norm_forward(norm, S, H, t, H * 384, 384, gains[i], None, t, H * 384, 384)
    q, k = mine[:, :, 0], mine[:, :, 1]
    h3.h3_rope(rope, S, pos, 0, q, q, H, k, k, H, H * 384, 384, H * 384, 384)
    ok()
    assert torch.equal(mine[:, :, 2], qkv[:, :, 2])
    a, b = f64(mine[:, :, :2]), f64(qkv[:, :, :2])
    # a rounding of the norm may fall to either side (one step, 2^-7 relative),
    # and moves both channels of its pair; then one rounding each
    size = np.abs(b) + np.abs(np.concatenate([b[..., 48:96], b[..., :48], 0 * b[..., 96:]], -1))
    assert (np.abs(a - b) <= 2.0 ** -6 * size).all()
    assert np.mean(a != b) < 0.02


# ---------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------

WIDTHS = [1, 2, 7, 8, 9, 64, 127, 128, 129, 256, 257, 500, 512, 1009, 1024, 1030, 2048, 2688, 4090, 5376, 6145, 8192]


def norm_rows(rows, heads, width, dtype, seed, gap=0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    unit = 16 // dtype.itemsize
    full = torch.full((rows, heads, (width + unit - 1) // unit * unit + gap), float("nan"), dtype=dtype)
    full[..., :width] = (mean + torch.randn(rows, heads, width, generator=g)).to(dtype)
    return full.cuda()


def run_norm(kind, dtype, rows, heads, width, pdtype=None, gain=True, bias=True, mean=0.0, gap=8, grads=True):
    tdtype, code, half = DTYPES[dtype]
    ptype, pcode, _ = DTYPES[pdtype or dtype]
    g = torch.Generator().manual_seed(width)
    x = norm_rows(rows, heads, width, tdtype, 1, gap, mean)
    dy = norm_rows(rows, heads, width, tdtype, 2, 2 * gap)
    gn = (1 + 0.3 * torch.randn(width, generator=g)).to(ptype).cuda() if gain else None
    bs = torch.randn(width, generator=g).to(ptype).cuda() if bias else None
    cfg = h3.make_norm_config(KINDS[kind], width, code, pcode)
    y, dx = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    h3.h3_norm_forward(cfg, rows, heads, x, x.stride(0), x.stride(1), gn, bs, y, y.stride(0), y.stride(1))
    dg, db = (torch.full((width,), 9.0, device="cuda") if grads else None for _ in range(2))
    ws = torch.empty(h3.h3_norm_backward_workspace_bytes(cfg, rows, heads), dtype=torch.uint8, device="cuda")
    h3.h3_norm_backward(cfg, rows, heads, x, x.stride(0), x.stride(1), gn, dy, dy.stride(0), dy.stride(1), dx,
                        dx.stride(0), dx.stride(1), dg, db, ws if grads else None)
    ok()
    what = f"{kind} {dtype} {rows}x{heads}x{width}"
    none = lambda t: None if t is None else f64(t)  # noqa: E731
    ref, bound = O.norm_forward(f64(x[..., :width]), kind, none(gn), none(bs), half=half)
    within(y[..., :width], ref, bound, what + " y")
    ref, bound = O.norm_backward(f64(x[..., :width]), f64(dy[..., :width]), kind, none(gn), half=half)
    within(dx[..., :width], ref["dx"], bound["dx"], what + " dx")
    if grads:
        within(dg, ref["dgain"], bound["dgain"], what + " dgain")
        within(db, ref["dbias"], bound["dbias"], what + " dbias")
    assert (y[..., width:] == 5.0).all() and (dx[..., width:] == 5.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_widths(kind, dtype, width):
    run_norm(kind, dtype, 19, 1, width)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows, heads, width", [(1, 1, 5376), (1, 1, 128), (2, 56, 128), (505, 1, 5376), (777, 3, 128),
                                                (2000, 1, 96), (1501, 2, 520)])
def test_norm_row_counts(kind, rows, heads, width):
    run_norm(kind, "bf16", rows, heads, width)


@pytest.mark.parametrize("gain, bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("pdtype", ["bf16", "fp32"])
def test_norm_parameters(gain, bias, pdtype):
    run_norm("layer", "bf16", 33, 2, 200, pdtype, gain, bias)
    run_norm("rms", "fp32", 33, 2, 200, pdtype, gain, bias, grads=False)


@pytest.mark.parametrize("dtype, mean", [("fp32", 1000.0), ("bf16", 50.0), ("fp32", -300.0)])
def test_layer_norm_of_rows_far_from_zero(dtype, mean):
    run_norm("layer", dtype, 21, 1, 1009, mean=mean)


def test_norm_constant_and_zero_rows():
    """A constant row has no spread and a zero row no size: xhat is 0 and
    1/sqrt(eps) scales the gradient; nothing becomes infinite."""
    cfg = h3.make_norm_config(h3.H3_NORM_LAYER, 136, h3.H3_FP32, h3.H3_FP32)
    x = torch.zeros(3, 1, 136, device="cuda")
    x[1] = 4.0
    x[2, 0, 0] = 1.0
    dy = torch.randn(3, 1, 136, generator=torch.Generator().manual_seed(1)).cuda()
    for kind in KINDS:
        cfg.kind = KINDS[kind]
        y, dx = torch.empty_like(x), torch.empty_like(x)
        h3.h3_norm_forward(cfg, 3, 1, x, 136, 136, None, None, y, 136, 136)
        h3.h3_norm_backward(cfg, 3, 1, x, 136, 136, None, dy, 136, 136, dx, 136, 136, None, None, None)
        ok()
        ref, bound = O.norm_forward(f64(x), kind, half=O.U32)
        within(y, ref, bound, kind)
        ref, bound = O.norm_backward(f64(x), f64(dy), kind, half=O.U32)
        within(dx, ref["dx"], bound["dx"], kind)


@pytest.mark.parametrize("width", [128, 1000, 5376])
def test_norm_in_place_repeat_and_one_parameter(width):
    rows = 300
    cfg = h3.make_norm_config(h3.H3_NORM_LAYER, width)
    x, dy = (norm_rows(rows, 1, width, torch.bfloat16, s) for s in (1, 2))
    gn = torch.rand(width, device="cuda").to(torch.bfloat16)
    st = x.stride(0)
    ws = torch.empty(h3.h3_norm_backward_workspace_bytes(cfg, rows, 1), dtype=torch.uint8, device="cuda")
    new = lambda: torch.empty(width, device="cuda")  # noqa: E731
    y, dx, dg, db = torch.empty_like(x), torch.empty_like(x), new(), new()
    h3.h3_norm_forward(cfg, rows, 1, x, st, st, gn, gn, y, st, st)
    h3.h3_norm_backward(cfg, rows, 1, x, st, st, gn, dy, st, st, dx, st, st, dg, db, ws)
    xx, yy, dg1, db1, dg2 = x.clone(), dy.clone(), new(), new(), new()
    h3.h3_norm_backward(cfg, rows, 1, x, st, st, gn, yy, st, st, yy, st, st, dg1, None, ws)     # dx over dy
    h3.h3_norm_backward(cfg, rows, 1, xx, st, st, gn, dy, st, st, xx, st, st, None, db1, ws)    # dx over x
    z = x.clone()
    h3.h3_norm_forward(cfg, rows, 1, z, st, st, gn, gn, z, st, st)
    ok()
    w = slice(0, width)
    assert torch.equal(yy[..., w], dx[..., w]) and torch.equal(xx[..., w], dx[..., w])
    assert torch.equal(dg1, dg) and torch.equal(db1, db) and torch.equal(z[..., w], y[..., w])


def test_norm_streams_and_graph():
    """Two streams at once with their own workspaces, and a captured pair of
    calls replayed with new contents."""
    rows, width = 400, 2688
    cfg = h3.make_norm_config(h3.H3_NORM_RMS, width)
    gn = torch.rand(width, device="cuda").to(torch.bfloat16)
    nws = h3.h3_norm_backward_workspace_bytes(cfg, rows, 1)

    def buffers(seed):
        x, dy = (norm_rows(rows, 1, width, torch.bfloat16, seed + s) for s in (0, 1))
        return (x, dy, torch.empty_like(x), torch.empty(width, device="cuda"), torch.empty(width, device="cuda"),
                torch.empty(nws, dtype=torch.uint8, device="cuda"))

    def go(b, stream=None):
        x, dy, dx, dg, db, ws = b
        h3.h3_norm_backward(cfg, rows, 1, x, width, width, gn, dy, width, width, dx, width, width, dg, db, ws, stream)
        return [t.clone() for t in (dx, dg, db)] if stream is None else None

    sets = [buffers(10), buffers(20)]
    want = [go(b) for b in sets]
    torch.cuda.synchronize()
    for b in sets:
        for t in b[2:5]:
            t.zero_()
    torch.cuda.synchronize()
    for b, s in zip(sets, [torch.cuda.Stream(), torch.cuda.Stream()]):
        go(b, s)
    torch.cuda.synchronize()
    for b, w in zip(sets, want):
        assert all(torch.equal(x, y) for x, y in zip(b[2:5], w))
    graph = torch.cuda.CUDAGraph()
    x, dy, dx, dg, db, ws = sets[0]
    with torch.cuda.graph(graph):
        h3.h3_norm_backward(cfg, rows, 1, x, width, width, gn, dy, width, width, dx, width, width, dg, db, ws)
    x.copy_(sets[1][0])
    dy.copy_(sets[1][1])
    graph.replay()
    ok()
    assert all(torch.equal(a, b) for a, b in zip((dx, dg, db), want[1]))


# ---------------------------------------------------------------------------
# together: the attention branch, forward and backward
# ---------------------------------------------------------------------------

def test_attention_branch_gradient():
    """y = x + attention branch, with the library's own forward calls (block
    norm, QKV projection, per-head norm, rotary positions, attention, output
    projection), then its gradient through the operators above, each stage
    against the oracle on the stage's own inputs, and the whole against the
    fp64 chain of the oracles."""
    S, H, D = 200, 2, 256
    g = torch.Generator().manual_seed(77)
    dev = lambda t: t.to(torch.bfloat16).cuda()  # noqa: E731
    x = dev(torch.randn(S, 1, D, generator=g))
    gain = dev(1 + 0.1 * torch.randn(D, generator=g))
    qk_gain = [dev(1 + 0.1 * torch.randn(128, generator=g)) for _ in range(2)]
    w_qkv = dev(torch.randn(H * 384, D, generator=g) / 16)
    w_o = dev(torch.randn(D, H * 128, generator=g) / 16)
    pos = torch.randint(0, 40, (S, 3), generator=g, dtype=torch.int32).cuda()
    dy = dev(torch.randn(S, D, generator=g))
    cn, cq = h3.make_norm_config(h3.H3_NORM_RMS, D), h3.make_norm_config(h3.H3_NORM_RMS, 128)
    cr = h3.make_rope_config(128, 3, 16)
    rs, hs = H * 384, 384
    new = lambda *shape: torch.empty(*shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731

    # forward
    hidden, raw, o = new(S, 1, D), new(S, H, 3, 128), new(S, H, 128)
    lse = torch.empty(H, S, device="cuda")
    h3.h3_norm_forward(cn, S, 1, x, D, D, gain, None, hidden, D, D)
    h3.h3_linear(S, H * 384, D, hidden, w_qkv, None, raw)
    qkv = raw.clone()
    for i in range(2):
        h3.h3_norm_forward(cq, S, H, raw[:, :, i], rs, hs, qk_gain[i], None, qkv[:, :, i], rs, hs)
    q, k, v = (qkv[:, :, i] for i in range(3))
    h3.h3_rope(cr, S, pos, h3.H3_ROPE_FORWARD, q, q, H, k, k, H, rs, hs, rs, hs)
    h3.h3_attention(S, H, q, k, v, rs, hs, o, lse)
    # backward
    d_o, d_qkv, d_raw, d_hidden, dx = new(S, H, 128), new(S, H, 3, 128), new(S, H, 3, 128), new(S, 1, D), new(S, 1, D)
    ws = torch.empty(max(h3.h3_attention_backward_workspace_bytes(S, H), h3.h3_norm_backward_workspace_bytes(cq, S, H),
                         h3.h3_norm_backward_workspace_bytes(cn, S, 1)), dtype=torch.uint8, device="cuda")
    d_gains = [torch.empty(128, device="cuda") for _ in range(2)]
    d_gain = torch.empty(D, device="cuda")
    h3.h3_linear(S, H * 128, D, dy, w_o.t().contiguous(), None, d_o)
    dq, dk, dv = (d_qkv[:, :, i] for i in range(3))
    h3.h3_attention_backward(S, H, q, k, v, rs, hs, o, d_o, lse, dq, dk, dv, rs, hs, ws)
    h3.h3_rope(cr, S, pos, h3.H3_ROPE_BACKWARD, dq, dq, H, dk, dk, H, rs, hs, rs, hs)
    for i in range(2):
        h3.h3_norm_backward(cq, S, H, raw[:, :, i], rs, hs, qk_gain[i], d_qkv[:, :, i], rs, hs, d_raw[:, :, i], rs, hs,
                            d_gains[i], None, ws)
    d_raw[:, :, 2].copy_(dv)
    h3.h3_linear(S, D, H * 384, d_raw, w_qkv.t().contiguous(), None, d_hidden)
    h3.h3_norm_backward(cn, S, 1, x, D, D, gain, d_hidden, D, D, dx, D, D, d_gain, None, ws)
    ok()

    # each stage on its own inputs (the stages after dq, dk were turned in place)
    table = O.rope_frequencies(3, 16)
    heads = [(f64(q[:, h]), f64(k[:, h]), f64(v[:, h]), f64(o[:, h]), f64(d_o[:, h]), f64(lse[h])) for h in range(H)]
    att = [O.attention_backward(*t) for t in heads]
    for i, name in ((2, "dv"),):
        for h in range(H):
            within(d_qkv[:, h, i], att[h][0][name], att[h][1][name], name)
    for i, name in ((0, "dq"), (1, "dk")):
        ref = np.stack([att[h][0][name] for h in range(H)], 1)
        bound = np.stack([att[h][1][name] for h in range(H)], 1)
        turned, b = O.rope(ref, pos.cpu().numpy(), table, backward=True)
        spread, _ = O.rope(bound, np.zeros((S, 3), int), table)
        other = np.concatenate([spread[..., 48:96], spread[..., :48], 0 * spread[..., 96:]], -1)
        within(d_qkv[:, :, i], turned, (spread + other) * (1 + 2 * O.HALF_BF16) + b + O.HALF_BF16 * np.abs(turned), name)
        ref, bound = O.norm_backward(f64(raw[:, :, i]), f64(d_qkv[:, :, i]), "rms", f64(qk_gain[i]))
        within(d_raw[:, :, i], ref["dx"], bound["dx"], name + " norm")
        within(d_gains[i], ref["dgain"], bound["dgain"], name + " gain")
    ref, bound = O.norm_backward(f64(x), f64(d_hidden), "rms", f64(gain))
    within(dx, ref["dx"], bound["dx"], "dx")
    within(d_gain, ref["dgain"], bound["dgain"], "gain")

    # the whole in fp64, without the roundings in between.  15 tensors are
    # rounded to bf16 on the way (each at most 2^-8 relative, in norm), and
    # every stage passes a relative error on with a factor of 2 at most: the
    # norm's projection and the rotation do not enlarge it, the products mix
    # independent errors, and P, dS carry those of q and k (scores of size 1).
    X, G, W, Wo = f64(x), f64(gain), f64(w_qkv), f64(w_o)
    hid, _ = O.norm_forward(X, "rms", G)
    r = (hid[:, 0] @ W.T).reshape(S, H, 3, 128)
    P = pos.cpu().numpy()
    QK = [O.rope(O.norm_forward(r[:, :, i], "rms", f64(qk_gain[i]))[0], P, table)[0] for i in range(2)]
    dO = (f64(dy) @ Wo).reshape(S, H, 128)
    d_r = np.empty_like(r)
    parts = []
    for h in range(H):
        oo, ll = O.attention_forward(QK[0][:, h], QK[1][:, h], r[:, h, 2])
        parts.append(O.attention_backward(QK[0][:, h], QK[1][:, h], r[:, h, 2], oo, dO[:, h], ll)[0])
    for i, name in ((0, "dq"), (1, "dk")):
        t, _ = O.rope(np.stack([p[name] for p in parts], 1), P, table, backward=True)
        d_r[:, :, i] = O.norm_backward(r[:, :, i], t, "rms", f64(qk_gain[i]))[0]["dx"]
    d_r[:, :, 2] = np.stack([p["dv"] for p in parts], 1)
    want = O.norm_backward(X, (d_r.reshape(S, -1) @ W).reshape(S, 1, D), "rms", G)[0]
    for got, ref in ((dx, want["dx"]), (d_gain, want["dgain"])):
        rel = np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)
        assert rel <= 15 * 2 * 2.0 ** -8, rel
