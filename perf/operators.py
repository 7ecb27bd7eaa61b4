"""Measured cases of the training-side operators: the attention gradient, rotary positions with their
gradient, and the row norms with theirs.

listed() and draw() give cases, prepare() makes a case's inputs on the GPU, run() makes one pass (in
elementary torch operations, or with `own` through the library's entry points), exact() gives the same
outputs from the definitions in 64 bits, work() counts what a pass cannot do without.
"""
from __future__ import annotations

import math

import torch

own = False

HEAD = 128                        # channels of an attention head
LARGEST_ATTENTION = 15860 ** 2 * 56   # row pairs times heads of the largest listed case
EXACT_ATTENTION = 4_000_000_000   # above this many row pairs times heads, 64 bits take too long


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # gradient of the attention core.  The tiny block's 72 rows: launch latency counts.
        {"name": "attention_backward tiny", "op": "attention_backward", "rows": 72, "heads": 4, "packed": True},
        # one full-width block over a short clip: a training step on 505 packed rows
        {"name": "attention_backward block", "op": "attention_backward", "rows": 505, "heads": 56, "packed": True},
        # separate q, k, v tensors of an odd number of heads, rows that end inside a tile
        {"name": "attention_backward ragged", "op": "attention_backward", "rows": 4099, "heads": 13, "packed": False},
        # the denoiser's long document: fine-tuning on, or guiding, an 864x480 clip of 141 frames
        {"name": "attention_backward long", "op": "attention_backward", "rows": 15860, "heads": 56, "packed": True},
        # the block norm over the long document
        {"name": "norm_forward long", "op": "norm_forward", "kind": "rms", "dtype": "bf16", "rows": 15860,
         "heads": 1, "width": 5376, "bias": False, "strided": False},
        # a layer norm of an FP32 module, its width no multiple of a vector
        {"name": "norm_forward odd", "op": "norm_forward", "kind": "layer", "dtype": "fp32", "rows": 257,
         "heads": 1, "width": 1009, "bias": True, "strided": False},
        # the block norm's gradient on a short clip
        {"name": "norm_backward block", "op": "norm_backward", "kind": "rms", "dtype": "bf16", "rows": 505,
         "heads": 1, "width": 5376, "bias": False, "strided": False},
        # a layer norm's gradient over the long document, gain and bias
        {"name": "norm_backward long", "op": "norm_backward", "kind": "layer", "dtype": "bf16", "rows": 15860,
         "heads": 1, "width": 5376, "bias": True, "strided": False},
        # the per-head Q norm's gradient on the q slots of packed q, k, v
        {"name": "norm_backward heads", "op": "norm_backward", "kind": "rms", "dtype": "bf16", "rows": 1824,
         "heads": 56, "width": 128, "bias": False, "strided": True},
        # three-axis positions on 96 of 128 channels of q and k, the long document
        {"name": "rope long", "op": "rope", "dtype": "bf16", "layout": "half", "axes": 3, "freqs": 16, "width": 128,
         "rows": 15860, "q_heads": 56, "k_heads": 56, "scaling": "none", "factor": 1.0, "scaled_axes": 7,
         "backward": False, "strided": True, "far": 1 << 10},
        # its gradient on a short clip whose time axis is stretched beyond the trained length
        {"name": "rope_backward block", "op": "rope", "dtype": "bf16", "layout": "half", "axes": 3, "freqs": 16,
         "width": 128, "rows": 505, "q_heads": 56, "k_heads": 56, "scaling": "linear", "factor": 4.0,
         "scaled_axes": 1, "backward": True, "strided": True, "far": 1 << 12},
        # one token far into a long context: shared key heads, pairs side by side, frequencies scaled by parts
        {"name": "rope token", "op": "rope", "dtype": "fp32", "layout": "interleaved", "axes": 1, "freqs": 32,
         "width": 80, "rows": 1, "q_heads": 32, "k_heads": 8, "scaling": "yarn", "factor": 32.0, "scaled_axes": 1,
         "backward": False, "strided": False, "far": 1 << 20},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention_backward", "attention_backward", "norm_forward", "norm_backward", "rope"])
    if op == "attention_backward":
        heads = rng.randint(1, 56)
        most = int(math.isqrt(LARGEST_ATTENTION // heads))
        # from two rows: the softmax over a single one is constant, and its gradient zero
        return {"op": op, "rows": _log_int(rng, 2, min(most, 16384)), "heads": heads, "packed": rng.random() < 0.5}
    if op == "rope":
        axes = rng.choice([1, 2, 3])
        freqs = rng.randint(2, 64 // axes)
        width = min(2 * axes * freqs + rng.choice([0, 0, 2, 16, 32]), 192)
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return {"op": op, "dtype": rng.choice(["bf16", "fp32"]), "layout": rng.choice(["half", "interleaved"]),
                "axes": axes, "freqs": freqs, "width": width, "rows": _log_int(rng, 1, 15000),
                "q_heads": rng.randint(1, 56), "k_heads": rng.choice([0, 1, 8, 56]), "scaling": scaling,
                "factor": 1.0 if scaling == "none" else float(rng.choice([2, 4, 32])),
                "scaled_axes": rng.randint(1, (1 << axes) - 1), "backward": rng.random() < 0.5,
                "strided": rng.random() < 0.5, "far": 1 << rng.randint(8, 24)}
    heads = rng.choice([1, 1, rng.randint(2, 56)])
    width = _log_int(rng, 32, 8192) if heads == 1 else rng.randint(32, 256)
    most = min(65536, 15860 * 5376 // (heads * width))
    return {"op": op, "kind": rng.choice(["rms", "layer"]), "dtype": rng.choice(["bf16", "fp32"]),
            "rows": _log_int(rng, 1, most), "heads": heads, "width": width,
            "bias": rng.random() < 0.5, "strided": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


def _padded(width, dtype):
    """Row length that keeps rows on 16-byte boundaries."""
    unit = 8 if dtype == torch.bfloat16 else 4
    return (width + unit - 1) // unit * unit


def _rows(shape, dtype, strided, g):
    """Seeded normal values [rows][heads][width]: a view into rows of their own, or (strided) into slots of
    three per head, as q is of packed q, k, v."""
    rows, heads, width = shape
    if strided:
        full = torch.empty(rows, heads, 3, _padded(width, dtype), dtype=dtype, device="cuda")
        view = full[:, :, 0, :width]
    else:
        full = torch.empty(rows, heads, _padded(width, dtype), dtype=dtype, device="cuda")
        view = full[:, :, :width]
    view.copy_(torch.randn(rows, heads, width, generator=g, device="cuda"))
    return view


def _rms_rows(x):
    return x / x.square().mean(-1, keepdim=True).sqrt()


def _prepare_attention(case, g):
    s, h = case["rows"], case["heads"]
    # q and k as the per-head norm leaves them (unit root mean square times learned gains near 1)
    gain = 1.0 + 0.1 * torch.randn(2, 1, 1, HEAD, generator=g, device="cuda")
    q = (_rms_rows(torch.randn(s, h, HEAD, generator=g, device="cuda")) * gain[0]).to(torch.bfloat16)
    k = (_rms_rows(torch.randn(s, h, HEAD, generator=g, device="cuda")) * gain[1]).to(torch.bfloat16)
    v = torch.randn(s, h, HEAD, generator=g, device="cuda").to(torch.bfloat16)
    d_o = torch.randn(s, h * HEAD, generator=g, device="cuda").to(torch.bfloat16)
    # what the forward pass leaves: its output and the logarithm of each row's sum
    qh, kh, vh = (t.float().transpose(0, 1) for t in (q, k, v))
    p = torch.matmul(qh, kh.transpose(1, 2)).mul_(1.0 / math.sqrt(HEAD))
    m = p.amax(-1, keepdim=True)
    p = p.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (m + total.log()).squeeze(-1).contiguous()
    o = (torch.matmul(p, vh) / total).transpose(0, 1).reshape(s, h * HEAD).to(torch.bfloat16)
    if case["packed"]:
        qkv = torch.stack([q, k, v], dim=2).contiguous()
        q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    return {"q": q, "k": k, "v": v, "o": o, "d_o": d_o, "lse": lse}


def _prepare_norm(case, g):
    dtype, width = _DTYPES[case["dtype"]], case["width"]
    shape = (case["rows"], case["heads"], width)
    state = {"x": _rows(shape, dtype, case["strided"], g)}
    if case["op"] == "norm_backward":
        state["dy"] = _rows(shape, dtype, case["strided"], g)
    state["gain"] = (1.0 + 0.1 * torch.randn(width, generator=g, device="cuda")).to(dtype)
    state["bias"] = (0.1 * torch.randn(width, generator=g, device="cuda")).to(dtype) if case["bias"] else None
    return state


def _prepare_rope(case, g):
    dtype, width, rows = _DTYPES[case["dtype"]], case["width"], case["rows"]
    pos = torch.randint(0, case["far"], (rows, case["axes"]), generator=g, device="cuda", dtype=torch.int32)
    q = _rows((rows, case["q_heads"], width), dtype, case["strided"], g)
    k = _rows((rows, case["k_heads"], width), dtype, case["strided"], g) if case["k_heads"] else None
    if k is not None and case["q_heads"] != case["k_heads"]:
        # q and k share their strides: rows of both in one buffer
        both = torch.cat([q, k], dim=1)
        buf = torch.zeros(rows, both.shape[1], _padded(width, dtype), dtype=dtype, device="cuda")
        buf[:, :, :width] = both
        q, k = buf[:, :case["q_heads"], :width], buf[:, case["q_heads"]:, :width]
    return {"q": q, "k": k, "pos": pos}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = {"attention_backward": _prepare_attention, "norm_forward": _prepare_norm,
            "norm_backward": _prepare_norm, "rope": _prepare_rope}[case["op"]]
    return {"case": case, **make(case, g)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"attention_backward": _own_attention, "norm_forward": _own_norm_forward,
                "norm_backward": _own_norm_backward, "rope": _own_rope}[op](state)
    return {"attention_backward": _plain_attention, "norm_forward": _plain_norm_forward,
            "norm_backward": _plain_norm_backward, "rope": _plain_rope}[op](state)


def _plain_attention(state):
    """P = exp(q k^T / sqrt(d) - lse); dV = P^T dO; dS = P (dO V^T - rowsum(dO O)) / sqrt(d); dQ = dS K;
    dK = dS^T Q."""
    s, h = state["case"]["rows"], state["case"]["heads"]
    heads = lambda t: t.reshape(s, h, HEAD).float().transpose(0, 1)  # noqa: E731
    q, k, v, o, d_o = (heads(state[n]) for n in ("q", "k", "v", "o", "d_o"))
    scale = 1.0 / math.sqrt(HEAD)
    p = torch.matmul(q, k.transpose(1, 2)).mul_(scale).sub_(state["lse"].unsqueeze(-1)).exp_()
    dv = torch.matmul(p.transpose(1, 2), d_o)
    ds = torch.matmul(d_o, v.transpose(1, 2)).sub_((d_o * o).sum(-1, keepdim=True)).mul_(p)
    del p
    dq = torch.matmul(ds, k).mul_(scale)
    dk = torch.matmul(ds.transpose(1, 2), q).mul_(scale)
    return {n: t.transpose(0, 1).to(torch.bfloat16) for n, t in (("dq", dq), ("dk", dk), ("dv", dv))}


def _normalised(x, kind):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    rstd = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return x * rstd, rstd


def _plain_norm_forward(state):
    xhat, _ = _normalised(state["x"].float(), state["case"]["kind"])
    y = xhat * state["gain"].float()
    if state["bias"] is not None:
        y = y + state["bias"].float()
    return {"y": y.to(state["x"].dtype)}


def _plain_norm_backward(state):
    """xhat the normalised row, w = dy gain: dx = rstd (w - mean(w) - xhat mean(w xhat)), the mean of w for the
    layer norm alone; dgain = sum of dy xhat over the rows, dbias = sum of dy."""
    kind = state["case"]["kind"]
    dy = state["dy"].float()
    xhat, rstd = _normalised(state["x"].float(), kind)
    w = dy * state["gain"].float()
    dx = w - xhat * (w * xhat).mean(-1, keepdim=True)
    if kind == "layer":
        dx = dx - w.mean(-1, keepdim=True)
    out = {"dx": (dx * rstd).to(state["x"].dtype), "dgain": (dy * xhat).sum((0, 1))}
    if state["bias"] is not None:
        out["dbias"] = dy.sum((0, 1))
    return out


def _frequencies(case):
    """Angle per position of each rotated pair, [axes][freqs] in 64 bits.  linear: positions divided by the
    factor; ntk: the base raised so that the lowest frequency is divided by the factor; yarn: frequencies that
    turn fewer than ALPHA times over the trained length divided, those that turn more than BETA times kept, a
    ramp between."""
    f = torch.arange(case["freqs"], dtype=torch.float64, device="cuda")
    base = THETA ** (-f / case["freqs"])
    s = case["factor"]
    if case["scaling"] == "linear":
        scaled = base / s
    elif case["scaling"] == "ntk":
        scaled = (THETA * s ** (case["freqs"] / (case["freqs"] - 1))) ** (-f / case["freqs"])
    elif case["scaling"] == "yarn":
        keep = ((TRAINED * base / (2 * math.pi) - ALPHA) / (BETA - ALPHA)).clamp(0, 1)
        scaled = base * keep + base / s * (1 - keep)
    else:
        scaled = base
    chosen = torch.tensor([(case["scaled_axes"] >> a) & 1 for a in range(case["axes"])], device="cuda") > 0
    return torch.where(chosen[:, None], scaled, base)


THETA, TRAINED, ALPHA, BETA = 10000.0, 4096, 1.0, 32.0


def _magnitude(case):
    return 1.25 if case["scaling"] == "yarn" else 1.0


def _pairs(t, case):
    half = case["axes"] * case["freqs"]
    if case["layout"] == "half":
        return t[..., :half], t[..., half:2 * half]
    return t[..., :2 * half:2], t[..., 1:2 * half:2]


def _rotated(t, cos, sin, case):
    out = t.clone()
    a, b = _pairs(t, case)
    to_a, to_b = _pairs(out, case)
    to_a.copy_(a * cos - b * sin)
    to_b.copy_(a * sin + b * cos)
    return out


def _plain_rope(state):
    case = state["case"]
    angle = (state["pos"].double().unsqueeze(-1) * _frequencies(case)).reshape(case["rows"], 1, -1)
    cos = (angle.cos() * _magnitude(case)).float()
    sin = (angle.sin() * (-_magnitude(case) if case["backward"] else _magnitude(case))).float()
    out = {"q": _rotated(state["q"].float(), cos, sin, case).to(state["q"].dtype)}
    if state["k"] is not None:
        out["k"] = _rotated(state["k"].float(), cos, sin, case).to(state["k"].dtype)
    return out


# ---------------------------------------------------------------------------
# one pass through the library; buffers, workspace and configuration are kept with the state, as a program
# that calls the operator every step keeps them
# ---------------------------------------------------------------------------

def _like_rows(t):
    """Output rows of t's shape on 16-byte boundaries."""
    rows, heads, width = t.shape
    return torch.empty(rows, heads, _padded(width, t.dtype), dtype=t.dtype, device="cuda")[:, :, :width]


def _own_attention(state):
    import audio_video_flow_gb300 as h3
    s, h = state["case"]["rows"], state["case"]["heads"]
    kept = state.get("own")
    if kept is None:
        grads = torch.empty(s, h, 3, HEAD, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(h3.h3_attention_backward_workspace_bytes(s, h), dtype=torch.uint8, device="cuda")
        kept = state["own"] = {"dq": grads[:, :, 0], "dk": grads[:, :, 1], "dv": grads[:, :, 2]}, ws
    out, ws = kept
    q = state["q"]
    h3.h3_attention_backward(s, h, q, state["k"], state["v"], q.stride(0), q.stride(1), state["o"], state["d_o"],
                             state["lse"], out["dq"], out["dk"], out["dv"], 3 * h * HEAD, 3 * HEAD, ws)
    return out


def _norm_config(case):
    import audio_video_flow_gb300 as h3
    kind = h3.H3_NORM_LAYER if case["kind"] == "layer" else h3.H3_NORM_RMS
    dtype = h3.H3_BF16 if case["dtype"] == "bf16" else h3.H3_FP32
    return h3.make_norm_config(kind, case["width"], dtype, dtype, EPS)


def _own_norm_forward(state):
    import audio_video_flow_gb300 as h3
    case, x = state["case"], state["x"]
    kept = state.get("own")
    if kept is None:
        kept = state["own"] = _norm_config(case), _like_rows(x)
    cfg, y = kept
    h3.h3_norm_forward(cfg, case["rows"], case["heads"], x, x.stride(0), x.stride(1), state["gain"], state["bias"],
                       y, y.stride(0), y.stride(1))
    return {"y": y}


def _own_norm_backward(state):
    import audio_video_flow_gb300 as h3
    case, x, dy = state["case"], state["x"], state["dy"]
    kept = state.get("own")
    if kept is None:
        cfg = _norm_config(case)
        ws = torch.empty(h3.h3_norm_backward_workspace_bytes(cfg, case["rows"], case["heads"]), dtype=torch.uint8,
                         device="cuda")
        out = {"dx": _like_rows(x), "dgain": torch.empty(case["width"], device="cuda")}
        if case["bias"]:
            out["dbias"] = torch.empty(case["width"], device="cuda")
        kept = state["own"] = cfg, out, ws
    cfg, out, ws = kept
    dx = out["dx"]
    h3.h3_norm_backward(cfg, case["rows"], case["heads"], x, x.stride(0), x.stride(1), state["gain"], dy,
                        dy.stride(0), dy.stride(1), dx, dx.stride(0), dx.stride(1), out["dgain"], out.get("dbias"), ws)
    return out


def _own_rope(state):
    import audio_video_flow_gb300 as h3
    case, q, k = state["case"], state["q"], state["k"]
    kept = state.get("own")
    if kept is None:
        scaling = {"none": h3.H3_ROPE_SCALE_NONE, "linear": h3.H3_ROPE_SCALE_LINEAR, "ntk": h3.H3_ROPE_SCALE_NTK,
                   "yarn": h3.H3_ROPE_SCALE_YARN}[case["scaling"]]
        cfg = h3.make_rope_config(
            case["width"], case["axes"], case["freqs"],
            layout=h3.H3_ROPE_HALF if case["layout"] == "half" else h3.H3_ROPE_INTERLEAVED,
            dtype=h3.H3_BF16 if case["dtype"] == "bf16" else h3.H3_FP32, theta=THETA, scaling=scaling,
            factor=case["factor"], scaled_axes=case["scaled_axes"], trained_length=TRAINED, alpha=ALPHA, beta=BETA,
            magnitude=_magnitude(case))
        heads = case["q_heads"] + case["k_heads"]
        both = torch.empty(case["rows"], heads, _padded(case["width"], q.dtype), dtype=q.dtype, device="cuda")
        out = {"q": both[:, :case["q_heads"], :case["width"]]}
        if k is not None:
            out["k"] = both[:, case["q_heads"]:, :case["width"]]
        kept = state["own"] = cfg, out
    cfg, out = kept
    direction = h3.H3_ROPE_BACKWARD if case["backward"] else h3.H3_ROPE_FORWARD
    to = out["q"]
    h3.h3_rope(cfg, case["rows"], state["pos"], direction, q, to, case["q_heads"], k, out.get("k"), case["k_heads"],
               q.stride(0), q.stride(1), to.stride(0), to.stride(1))
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_frequency(case, axis, f):
    """Radians per position of frequency f of an axis."""
    n, s, scaling = case["freqs"], case["factor"], case["scaling"]
    omega = math.exp(-math.log(THETA) * f / n)
    if scaling == "none" or not case["scaled_axes"] >> axis & 1:
        return omega
    if scaling == "linear":
        return omega / s
    if scaling == "ntk":
        return omega * s ** (-f / (n - 1))
    rounds = TRAINED * omega / (2 * math.pi)
    keep = min(1.0, max(0.0, (rounds - ALPHA) / (BETA - ALPHA)))
    return omega * (keep + (1.0 - keep) / s)


def exact(case, seed):
    if case["op"] == "attention_backward" and case["rows"] ** 2 * case["heads"] > EXACT_ATTENTION:
        return None
    state = prepare(case, seed)
    d = {n: t.double() if torch.is_tensor(t) else t for n, t in state.items()}
    if case["op"] == "attention_backward":
        per_head = (case["rows"], case["heads"], HEAD)
        q, k, v, o, d_o = (d[n].reshape(per_head) for n in ("q", "k", "v", "o", "d_o"))
        scale = HEAD ** -0.5
        p = torch.exp(torch.einsum("ihc,jhc->hij", q, k) * scale - d["lse"][:, :, None])
        delta = torch.einsum("ihc,ihc->hi", d_o, o)
        ds = p * (torch.einsum("ihc,jhc->hij", d_o, v) - delta[:, :, None]) * scale
        return {"dq": torch.einsum("hij,jhc->ihc", ds, k), "dk": torch.einsum("hij,ihc->jhc", ds, q),
                "dv": torch.einsum("hij,ihc->jhc", p, d_o)}
    if case["op"] == "rope":
        # every rotated pair's two channels as one complex number, turned by its own angle
        out, half = {}, case["axes"] * case["freqs"]
        omega = torch.tensor([_exact_frequency(case, a, f) for a in range(case["axes"]) for f in range(case["freqs"])],
                             dtype=torch.float64, device="cuda")
        axis = torch.arange(half, device="cuda") // case["freqs"]
        turns = d["pos"][:, axis] * omega * (-1.0 if case["backward"] else 1.0)
        unit = torch.polar(torch.full_like(turns, 1.25 if case["scaling"] == "yarn" else 1.0), turns)
        first = torch.arange(half, device="cuda")
        first, second = (first, first + half) if case["layout"] == "half" else (2 * first, 2 * first + 1)
        for name in ("q", "k"):
            if d[name] is None:
                continue
            z = torch.complex(d[name][..., first], d[name][..., second]) * unit[:, None, :]
            y = d[name].clone()
            y[..., first], y[..., second] = z.real, z.imag
            out[name] = y
        return out
    x, gain = d["x"], d["gain"]
    centre = x.mean(-1, keepdim=True) if case["kind"] == "layer" else torch.zeros_like(x[..., :1])
    spread = ((x - centre) ** 2).mean(-1, keepdim=True) + EPS
    xhat = (x - centre) / spread.sqrt()
    if case["op"] == "norm_forward":
        return {"y": xhat * gain + (d["bias"] if d["bias"] is not None else 0.0)}
    # the chain rule through the spread and, for the layer norm, the centre
    dy = d["dy"]
    dxhat = dy * gain
    dspread = (dxhat * (x - centre)).sum(-1, keepdim=True) * -0.5 * spread ** -1.5
    dx = dxhat / spread.sqrt() + dspread * 2.0 * (x - centre) / case["width"]
    if case["kind"] == "layer":
        dx = dx - dx.mean(-1, keepdim=True)
    out = {"dx": dx, "dgain": (dy * xhat).sum((0, 1))}
    if d["bias"] is not None:
        out["dbias"] = dy.sum((0, 1))
    return out


# ---------------------------------------------------------------------------
# work of one pass
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "attention_backward":
        s, h = case["rows"], case["heads"]
        # reads q, k, v, o, dO and lse, writes dq, dk, dv; five products of s x s x 128
        return {"bytes": s * h * (HEAD * 2 * 8 + 4), "flops": 10 * s * s * h * HEAD}
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        heads = case["q_heads"] + case["k_heads"]
        n = case["rows"] * heads
        return {"bytes": n * case["width"] * 2 * size + case["rows"] * case["axes"] * 4,
                "flops": n * case["axes"] * case["freqs"] * 6}
    n = case["rows"] * case["heads"] * case["width"]
    vectors = case["width"] * (1 + bool(case["bias"]))
    if case["op"] == "norm_forward":
        return {"bytes": 2 * n * size + vectors * size, "flops": 6 * n}
    return {"bytes": 3 * n * size + case["width"] * size + vectors * 4, "flops": 14 * n}
