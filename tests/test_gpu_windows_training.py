"""The windowed attention and its gradient as a training step runs them: the gradient call takes the output and the
log-sum-exp that the forward call left, and its results are those of the formulas in 64 bits."""
import numpy as np
import pytest
import torch

from oracle import h3_window_oracle as O
from oracle.h3_train_oracle import SQRT_D
from test_gpu_windows import draw, f64, ok, run_backward, run_window, window_case, within

pytestmark = pytest.mark.gpu


def exact(qs, k, v, d_os, mask):
    """The query heads of one KV head: ([dq], dk, dv) from the exact output and log-sum-exp, and the bounds of the two
    calls one after the other: the gradient's own, and what the forward's bounds on o and lse add to it.  With lse off
    by b_l, P is off by expm1(b_l) of itself; with o off by b_o, dS by P |dO| b_o besides."""
    outs = [O.forward(q, k, v, mask) for q in qs]
    grads, (b_dqs, b_dk, b_dv) = O.backward(qs, k, v, [o for (o, _), _ in outs], d_os, [lse for (_, lse), _ in outs], mask)
    b_dqs, b_dk, b_dv = list(b_dqs), b_dk.copy(), b_dv.copy()
    for i, (q, d_o, ((o, lse), (b_o, b_l))) in enumerate(zip(qs, d_os, outs)):
        p = np.where(mask, np.exp(np.where(mask, q @ k.T / SQRT_D - lse[:, None], -np.inf)), 0.0)
        ds = np.abs(p * (d_o @ v.T - (d_o * o).sum(axis=1, keepdims=True)))
        e_p = p * np.expm1(b_l)[:, None]
        e_ds = ds * np.expm1(b_l)[:, None] + (p + e_p) * (np.abs(d_o) * b_o).sum(axis=1, keepdims=True)
        # (the roundings that the gradient's own bound counts also fall on these: 2^-8 each of e_ds, e_p and the results)
        b_dqs[i] = b_dqs[i] + e_ds @ np.abs(k) / SQRT_D * (1 + 2.0 ** -6)
        b_dk += e_ds.T @ np.abs(q) / SQRT_D * (1 + 2.0 ** -6)
        b_dv += e_p.T @ np.abs(d_o) * (1 + 2.0 ** -6)
    return grads, (b_dqs, b_dk, b_dv)


@pytest.mark.parametrize("S, H, Hk, w", [
    (1, 2, 1, dict(right=0)),
    (72, 4, 4, dict(left=1, right=0, n_first=8, unit=16, origin=8)),
    (300, 6, 2, dict(left=70, right=9, n_first=3)),
    (700, 6, 3, dict()),                           # units of one tile that several CTAs share
    (1100, 4, 1, dict(right=0))])                  # and key tiles of the gradient in pieces
def test_forward_and_gradient(S, H, Hk, w):
    q, k, v = window_case(S, H, Hk, S + 3)
    d_o = draw(S, H, torch.Generator().manual_seed(S)).contiguous()
    o, lse = run_window(w, q, k, v)
    dq, dk, dv = run_backward(w, q, k, v, o, lse, d_o)
    ok()
    mask = O.visible(np.arange(S), S, **w)
    for a in range(Hk):
        heads = range(a * H // Hk, (a + 1) * H // Hk)
        (rq, rk, rv), (bq, bk, bv) = exact([f64(q[:, h]) for h in heads], f64(k[:, a]), f64(v[:, a]),
                                           [f64(d_o[:, h]) for h in heads], mask)
        for i, h in enumerate(heads):
            within(dq[:, h], rq[i], bq[i], f"head {h} dq")
        within(dk[:, a], rk, bk, f"kv head {a} dk")
        within(dv[:, a], rv, bv, f"kv head {a} dv")
