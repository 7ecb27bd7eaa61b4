"""Plain fp64 numpy oracle of the windowed and cached attention: masks, forward,
gradient, the weight that each key collects, and eviction by it.  Test
infrastructure only; shares no code with the CUDA path.

Bounds as in h3_train_oracle: sums of |partial error| over the terms of each
element, u = 2^-24 the half step of fp32, 2^-8 that of bf16."""
from __future__ import annotations

import numpy as np

from .h3_train_oracle import HALF_BF16, SQRT_D, U32

EXP = 2.0 ** -21      # relative error of an exponential or a logarithm's argument


def visible(rows, keys, left=-1, right=-1, n_first=0, unit=1, origin=0):
    """[len(rows)][keys]: what the rows at these positions see, from the definition."""
    unit_of = lambda i: np.floor((np.asarray(i, np.float64) - origin) / unit)  # noqa: E731
    ui, uj = unit_of(rows)[:, None], unit_of(np.arange(keys))[None, :]
    seen = np.ones((len(rows), keys), bool)
    if left >= 0:
        seen = (uj >= ui - left) | (np.arange(keys)[None, :] < n_first)
    if right >= 0:
        seen &= uj <= ui + right
    return seen


def _exponent_error(q, k, s, shift):
    """Error of s - shift in fp32: the dot product of 128 terms, the scaling and the difference."""
    return 130 * U32 * (np.abs(q) @ np.abs(k).T) / SQRT_D + 4 * U32 * (np.abs(s) + np.abs(shift))


def forward(q, k, v, mask):
    """One head: q [R][128], k, v [N][128] -> (o, lse), (bounds of both).  The running maximum that is subtracted
    lags the true one by at most 8 log 2; P is rounded to bf16 before its product and not in the sum."""
    n = k.shape[0]
    s = q @ k.T / SQRT_D
    masked = np.where(mask, s, -np.inf)
    m = masked.max(axis=1, keepdims=True)
    e = np.exp(masked - m)
    t = e.sum(axis=1, keepdims=True)
    p = e / t
    lse = (m + np.log(t))[:, 0]
    o = p @ v
    span = np.abs(np.where(mask, s, 0)).max(axis=1, keepdims=True) + 6
    rel_p = np.where(mask, np.expm1(_exponent_error(q, k, s, span)) + EXP, 0.0)
    # maxima that moved on rescale by an exponential each: at most one per key tile
    sums = (n + 32) * U32 + (n // 128 + 2) * EXP
    rel_l = (p * rel_p).sum(axis=1, keepdims=True) + sums
    e_o = (p * (rel_p + HALF_BF16 * (1 + rel_p) + sums)) @ np.abs(v) + rel_l * (p @ np.abs(v))
    bound_o = e_o * (1 + HALF_BF16 + rel_l) + HALF_BF16 * np.abs(o) + 1e-38
    # log2 of the sum and the maximum's scaling back
    bound_lse = (rel_l * 1.01)[:, 0] + 8 * U32 * (np.abs(lse) + span[:, 0] + np.abs(np.log(t))[:, 0]) + EXP
    return (o, lse), (bound_o, bound_lse)


def backward(qs, k, v, os, d_os, lses, mask):
    """The query heads of one KV head (lists): ([dq], dk, dv) and their bounds.  Counted as for the unmasked gradient;
    the accumulators of dk and dv run over the heads."""
    n = k.shape[0]
    dqs, b_dqs = [], []
    dk = dv = b_dk = b_dv = 0.0
    acc, acc_kv = (n + 2) * U32, (len(qs) * n + 2) * U32
    ak, av = np.abs(k), np.abs(v)
    for q, o, d_o, lse in zip(qs, os, d_os, lses):
        s = q @ k.T / SQRT_D
        p = np.where(mask, np.exp(np.where(mask, s - lse[:, None], -np.inf)), 0.0)
        dp = d_o @ v.T
        delta = (d_o * o).sum(axis=1, keepdims=True)
        ds = p * (dp - delta)
        rel_p = np.where(mask, np.expm1(_exponent_error(q, k, s, lse[:, None])) + EXP, 0.0)
        ad, aq = np.abs(d_o), np.abs(q)
        d_ds = np.abs(ds) * rel_p + p * (1 + rel_p) * 130 * U32 * (ad @ av.T + (ad * np.abs(o)).sum(axis=1, keepdims=True))
        e_ds = d_ds * (1 + HALF_BF16) + np.abs(ds) * HALF_BF16
        e_p = p * (rel_p * (1 + HALF_BF16) + HALF_BF16)
        dq = ds @ k / SQRT_D
        dqs.append(dq)
        b = (e_ds * (1 + acc) + np.abs(ds) * acc) @ ak / SQRT_D
        b_dqs.append(b * (1 + HALF_BF16) + HALF_BF16 * np.abs(dq) + 1e-38)
        dk = dk + ds.T @ q / SQRT_D
        dv = dv + p.T @ d_o
        b_dk = b_dk + (e_ds * (1 + acc_kv) + np.abs(ds) * acc_kv).T @ aq / SQRT_D
        b_dv = b_dv + (e_p * (1 + acc_kv) + p * acc_kv).T @ ad
    rounded = lambda b, r: b * (1 + HALF_BF16) + HALF_BF16 * np.abs(r) + 1e-38  # noqa: E731
    return (dqs, dk, dv), (b_dqs, rounded(b_dk, dk), rounded(b_dv, dv))


def collected(qs, k, lses, mask):
    """Sum over rows and the query heads of one KV head of exp(s - lse), visible: [N] and its bound."""
    total, bound, n = 0.0, 0.0, 0
    for q, lse in zip(qs, lses):
        s = q @ k.T / SQRT_D
        p = np.where(mask, np.exp(np.where(mask, s - lse[:, None], -np.inf)), 0.0)
        rel = np.expm1(_exponent_error(q, k, s, lse[:, None])) + EXP
        total = total + p.sum(axis=0)
        bound = bound + (p * rel).sum(axis=0)
        n += len(lse)
    return total, bound + (n + 4) * U32 * total


def kept_slots(weights, budget, n_first, n_recent):
    """Slots of one sequence and head that stay, ascending; weights [n] fp32."""
    n = len(weights)
    if n <= budget:
        return np.arange(n)
    middle = np.arange(n_first, n - n_recent)
    w = np.where(np.isnan(weights[middle]), -np.inf, weights[middle].astype(np.float64))
    # a NaN is below minus infinity, which it is only compared with
    order = middle[np.lexsort((middle, np.isnan(weights[middle]), -w))]
    best = order[:budget - n_first - n_recent]
    return np.sort(np.concatenate([np.arange(n_first), best, np.arange(n - n_recent, n)])).astype(np.int64)
