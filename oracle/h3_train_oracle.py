"""Plain fp64 numpy oracle of the training-side operators: the gradient of the
attention core, rotary positions in their general form, and the layer and RMS
norms with their gradients.  Test infrastructure only; shares no code with the
CUDA path.

Beside each result it gives an elementwise error bound for an evaluation that
computes in fp32, rounds the stated intermediates and rounds the result once:
the bounds are sums of |partial error| over the terms that make up the element,
with u = 2^-24 the half step of fp32 and `half` the half step of the result's
type (2^-8 for bf16, u for fp32)."""
from __future__ import annotations

import math

import numpy as np

U32 = 2.0 ** -24
HALF_BF16 = 2.0 ** -8
SQRT_D = math.sqrt(128.0)
TWO_PI = 2 * np.longdouble("3.14159265358979323846264338327950288")


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def attention_forward(q, k, v):
    """One head: q, k, v [S][128] -> o [S][128], lse [S]."""
    s = q @ k.T / SQRT_D
    m = s.max(axis=1, keepdims=True)
    e = np.exp(s - m)
    t = e.sum(axis=1, keepdims=True)
    return e @ v / t, (m + np.log(t))[:, 0]


def attention_backward(q, k, v, o, d_o, lse):
    """One head, from the given o and lse.  Returns ({dq, dk, dv}, {their
    elementwise bounds}).

    Errors counted: every fp32 dot product of n terms is within n u of the sum
    of its absolute terms; the exponent s - lse is within e_z = 130 u (|q|.|k|)
    / sqrt(d) + 4 u |lse| + 4 u |s|, so P is off by a factor exp(e_z), plus 2^-21 for
    the exponential itself; P and dS are rounded to bf16 (2^-8) before their
    products."""
    n = q.shape[0]
    s = q @ k.T / SQRT_D
    p = np.exp(s - lse[:, None])
    dp = d_o @ v.T
    delta = (d_o * o).sum(axis=1, keepdims=True)
    ds = p * (dp - delta)
    out = {"dq": ds @ k / SQRT_D, "dk": ds.T @ q / SQRT_D, "dv": p.T @ d_o}

    aq, ak, av, ad = np.abs(q), np.abs(k), np.abs(v), np.abs(d_o)
    e_z = 130 * U32 * (aq @ ak.T) / SQRT_D + 4 * U32 * (np.abs(lse)[:, None] + np.abs(s))
    rel_p = np.expm1(e_z) + 2.0 ** -21
    # dS before its rounding: P's relative error, and the errors of dP and D
    d_ds = np.abs(ds) * rel_p + p * (1 + rel_p) * 130 * U32 * (ad @ av.T + (ad * np.abs(o)).sum(axis=1, keepdims=True))
    e_ds = d_ds * (1 + HALF_BF16) + np.abs(ds) * HALF_BF16
    e_p = p * (rel_p * (1 + HALF_BF16) + HALF_BF16)
    acc = (n + 2) * U32
    rounded = lambda b, r: b * (1 + HALF_BF16) + np.abs(r) * HALF_BF16 + 1e-38  # noqa: E731
    bound = {"dq": rounded((e_ds * (1 + acc) + np.abs(ds) * acc) @ ak / SQRT_D, out["dq"]),
             "dk": rounded((e_ds * (1 + acc) + np.abs(ds) * acc).T @ aq / SQRT_D, out["dk"]),
             "dv": rounded((e_p * (1 + acc) + p * acc).T @ ad, out["dv"])}
    return out, bound


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

def rope_frequencies(n_axes, n_freqs, theta=10000.0, scaling="none", factor=1.0, scaled_axes=None,
                     trained_length=1.0, alpha=1.0, beta=32.0):
    """Radians per position, [n_axes][n_freqs], in extended precision (positions
    go to 2^31)."""
    ext = np.longdouble
    theta, factor = ext(theta), ext(factor)
    table = np.empty((n_axes, n_freqs), ext)
    for a in range(n_axes):
        scaled = scaling != "none" and (scaled_axes is None or (scaled_axes >> a) & 1)
        for f in range(n_freqs):
            w = theta ** (-ext(f) / n_freqs)
            if scaled and scaling == "linear":
                w /= factor
            elif scaled and scaling == "ntk":
                w = (theta * factor ** (ext(n_freqs) / (n_freqs - 1))) ** (-ext(f) / n_freqs)
            elif scaled and scaling == "yarn":
                g = min(max((trained_length * w / TWO_PI - alpha) / (beta - alpha), ext(0)), ext(1))
                w = g * w + (1 - g) * w / factor
            table[a, f] = w
    return table


def rope(x, pos, table, layout="half", magnitude=1.0, backward=False, half=HALF_BF16):
    """x [S][H][width], pos [S][n_axes] -> (result, bound).  Errors counted: the
    sine and cosine within 2^-21 (the angle's last bits and the function's),
    three fp32 roundings, one rounding to the result."""
    n_axes, n_freqs = table.shape
    pairs = n_axes * n_freqs
    if layout == "half":
        i0, i1 = np.arange(pairs), np.arange(pairs) + pairs
    else:
        i0, i1 = 2 * np.arange(pairs), 2 * np.arange(pairs) + 1
    # the angle reduced in extended precision: positions go to 2^31
    turns = pos.astype(np.longdouble)[:, :, None] * (np.asarray(table, np.longdouble) / TWO_PI)
    angle = ((turns - np.round(turns)) * TWO_PI).astype(np.float64).reshape(len(pos), 1, pairs)
    c, s = magnitude * np.cos(angle), (-magnitude if backward else magnitude) * np.sin(angle)
    out, bound = x.copy(), np.zeros_like(x)
    out[..., i0] = x[..., i0] * c - x[..., i1] * s
    out[..., i1] = x[..., i0] * s + x[..., i1] * c
    e = magnitude * (2.0 ** -21 + 4 * U32) * (np.abs(x[..., i0]) + np.abs(x[..., i1]))
    bound[..., i0] = e * (1 + half) + half * np.abs(out[..., i0])
    bound[..., i1] = e * (1 + half) + half * np.abs(out[..., i1])
    return out, bound + 1e-38 * (bound > 0)


# ---------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------

# A sum over a row of up to 8192 values: at most 32 in one thread's chain, 5
# butterfly levels and 8 warps, so within 48 u of the sum of absolute values;
# doubled for the products and the divisions around it.
ROW_SUM = 96 * U32


def _row_statistics(x, kind, eps):
    c = x - x.mean(-1, keepdims=True) if kind == "layer" else x
    r = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    # error of c (the mean's and the subtraction's), relative error of r,
    # absolute error of xhat
    e_c = ROW_SUM * (np.abs(x).mean(-1, keepdims=True) + np.abs(x)) if kind == "layer" else np.zeros_like(x)
    e_r = ROW_SUM + (np.abs(c) * e_c).mean(-1, keepdims=True) * r * r + (e_c * e_c).mean(-1, keepdims=True) * r * r
    e_xhat = e_c * r * (1 + e_r) + np.abs(c) * r * (e_r + 4 * U32)
    return c * r, r, e_xhat, e_r


def norm_forward(x, kind, gain=None, bias=None, eps=1e-5, half=HALF_BF16):
    """x [rows][heads][width] -> (y, bound)."""
    g = 1.0 if gain is None else gain
    b = np.zeros(x.shape[-1]) if bias is None else bias
    xhat, _, e_xhat, _ = _row_statistics(x, kind, eps)
    y = xhat * g + b
    e = np.abs(g) * (e_xhat * (1 + 2 * U32) + np.abs(xhat) * 2 * U32) + U32 * np.abs(b) + U32 * np.abs(y)
    return y, e * (1 + half) + half * np.abs(y) + 1e-38


def norm_backward(x, dy, kind, gain=None, eps=1e-5, half=HALF_BF16):
    """x, dy [rows][heads][width] -> ({dx, dgain, dbias}, {bounds})."""
    g = 1.0 if gain is None else gain
    mean = lambda t: t.mean(-1, keepdims=True)  # noqa: E731
    xhat, r, e_xhat, e_r = _row_statistics(x, kind, eps)
    w = dy * g
    m1 = mean(w * xhat)
    m0 = mean(w) if kind == "layer" else np.zeros_like(m1)
    inner = w - xhat * m1 - m0
    dx = r * inner
    aw = np.abs(w)
    e_m1 = mean(aw * e_xhat) + 2 * ROW_SUM * mean(np.abs(w * xhat)) + np.abs(m1) * e_r
    e_m0 = ROW_SUM * mean(aw) if kind == "layer" else 0.0
    e_inner = 4 * U32 * (aw + np.abs(xhat * m1) + np.abs(m0)) + e_xhat * (np.abs(m1) + e_m1) + np.abs(xhat) * e_m1 + e_m0
    e_dx = r * (1 + e_r) * e_inner + np.abs(dx) * (e_r + 4 * U32)
    n = x.shape[0] * x.shape[1]
    total = (n + 4) * U32
    out = {"dx": dx, "dgain": (dy * xhat).sum((0, 1)), "dbias": dy.sum((0, 1))}
    bound = {"dx": e_dx * (1 + half) + half * np.abs(dx) + 1e-38,
             "dgain": ((np.abs(dy) * e_xhat).sum((0, 1)) + total * np.abs(dy * xhat).sum((0, 1))) * (1 + total) + 1e-38,
             "dbias": total * np.abs(dy).sum((0, 1)) + 1e-38}
    return out, bound
