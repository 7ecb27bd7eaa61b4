"""Pins of the training-side oracle against facts that do not come from it:
differences of the forward functions, invariants, closed forms."""
import numpy as np
import pytest

from oracle import h3_train_oracle as O


def _difference(f, x, direction, h=1e-5):
    return (f(x + h * direction) - f(x - h * direction)) / (2 * h)


@pytest.mark.parametrize("n", [1, 2, 5, 17])
def test_attention_gradient_against_differences(rng, n):
    q, k, v, weight = (rng.standard_normal((n, 128)) for _ in range(4))
    o, lse = O.attention_forward(q, k, v)
    grads, _ = O.attention_backward(q, k, v, o, weight, lse)
    args = {"dq": q, "dk": k, "dv": v}
    for name, x in args.items():
        direction = rng.standard_normal(x.shape)
        loss = lambda t: (O.attention_forward(*(t if a == name else args[a] for a in ("dq", "dk", "dv")))[0]  # noqa: E731
                          * weight).sum()
        want = _difference(loss, x, direction)
        got = (grads[name] * direction).sum()
        # differences of a function of size |want|: h^2 third derivatives and eps / h
        assert abs(got - want) <= 1e-6 * (np.abs(grads[name] * direction).sum() + 1.0), name


def test_attention_gradient_of_one_row_and_of_equal_scores(rng):
    # one row: the softmax is constant, so dq = dk = 0 and dv = dO
    q, k, v, g = (rng.standard_normal((1, 128)) for _ in range(4))
    o, lse = O.attention_forward(q, k, v)
    d, _ = O.attention_backward(q, k, v, o, g, lse)
    assert np.abs(d["dq"]).max() < 1e-12 and np.abs(d["dk"]).max() < 1e-12
    np.testing.assert_allclose(d["dv"], g, rtol=1e-12)
    # q = 0: uniform probabilities
    n = 9
    k, v, g = (rng.standard_normal((n, 128)) for _ in range(3))
    o, lse = O.attention_forward(np.zeros((n, 128)), k, v)
    d, _ = O.attention_backward(np.zeros((n, 128)), k, v, o, g, lse)
    np.testing.assert_allclose(lse, np.log(n))
    np.testing.assert_allclose(d["dv"], np.tile(g.mean(0), (n, 1)), rtol=1e-12, atol=1e-14)
    assert np.abs(d["dk"]).max() == 0.0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_turns_pairs(rng, layout):
    table = O.rope_frequencies(2, 3, theta=100.0)
    x = rng.standard_normal((5, 2, 16))
    pos = rng.integers(-50, 50, (5, 2))
    y, _ = O.rope(x, pos, table, layout)
    back, _ = O.rope(y, pos, table, layout, backward=True)
    np.testing.assert_allclose(back, x, atol=1e-14)
    np.testing.assert_array_equal(y[..., 12:], x[..., 12:])
    np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    zero, _ = O.rope(x, np.zeros_like(pos), table, layout)
    np.testing.assert_array_equal(zero, x)
    # scores depend on the difference of positions alone
    q, k = rng.standard_normal((2, 1, 1, 16))
    score = lambda i, j: (O.rope(q, np.array([[i, i]]), table, layout)[0]  # noqa: E731
                          * O.rope(k, np.array([[j, j]]), table, layout)[0]).sum()
    assert abs(score(7, 3) - score(104, 100)) < 1e-12
    # the pair of frequency 0 turns by the position itself
    i1 = 6 if layout == "half" else 1
    e = np.zeros((1, 1, 16))
    e[..., 0] = 1.0
    y, _ = O.rope(e, np.array([[2, 0]]), table, layout)
    np.testing.assert_allclose([y[0, 0, 0], y[0, 0, i1]], [np.cos(2), np.sin(2)])


def test_rope_gradient_is_the_transpose(rng):
    table = O.rope_frequencies(1, 4)
    x, g = rng.standard_normal((2, 3, 1, 8))
    pos = rng.integers(0, 100, (3, 1))
    y, _ = O.rope(x, pos, table, magnitude=1.5)
    dx, _ = O.rope(g, pos, table, magnitude=1.5, backward=True)
    np.testing.assert_allclose((y * g).sum(), (x * dx).sum())


def test_rope_scalings():
    plain = O.rope_frequencies(2, 8)
    lin = O.rope_frequencies(2, 8, scaling="linear", factor=4.0, scaled_axes=1)
    np.testing.assert_allclose(np.float64(lin[0]), np.float64(plain[0]) / 4)
    np.testing.assert_array_equal(lin[1], plain[1])
    ntk = O.rope_frequencies(1, 8, scaling="ntk", factor=4.0)
    np.testing.assert_allclose(float(ntk[0, 0]), 1.0)
    np.testing.assert_allclose(float(ntk[0, -1]), float(plain[0, -1]) / 4)
    yarn = O.rope_frequencies(1, 64, scaling="yarn", factor=8.0, trained_length=4096.0)
    plain = O.rope_frequencies(1, 64)
    ratio = np.float64(yarn / plain)[0]
    assert ratio[0] == 1.0 and abs(ratio[-1] - 1 / 8) < 1e-12 and (np.diff(ratio) <= 1e-15).all()
    turns = 4096 * np.float64(plain[0]) / (2 * np.pi)
    mid = (turns > 1) & (turns < 32)
    g = (turns[mid] - 1) / 31
    np.testing.assert_allclose(ratio[mid], g + (1 - g) / 8)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_moments_and_invariance(rng, kind):
    x = rng.standard_normal((4, 2, 33)) * 3 + 1
    y, _ = O.norm_forward(x, kind, eps=1e-12)
    np.testing.assert_allclose((y ** 2).mean(-1), 1.0)
    if kind == "layer":
        np.testing.assert_allclose(y.mean(-1), 0.0, atol=1e-12)
        np.testing.assert_allclose(O.norm_forward(x + 5.0, kind, eps=1e-12)[0], y, atol=1e-10)
    np.testing.assert_allclose(O.norm_forward(2 * x, kind, eps=1e-12)[0], y, atol=1e-10)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("width", [1, 2, 13])
def test_norm_gradients_against_differences(rng, kind, width):
    x, dy, dirx = rng.standard_normal((3, 5, 2, width))
    gain, bias, dirg = rng.standard_normal((3, width))
    grads, _ = O.norm_backward(x, dy, kind, gain)
    checks = [("dx", lambda t: O.norm_forward(t, kind, gain, bias)[0], x, dirx),
              ("dgain", lambda t: O.norm_forward(x, kind, t, bias)[0], gain, dirg),
              ("dbias", lambda t: O.norm_forward(x, kind, gain, t)[0], bias, dirg)]
    for name, f, at, direction in checks:
        want = _difference(lambda t: (f(t) * dy).sum(), at, direction, 1e-6)
        got = (grads[name] * direction).sum()
        # second-order differences: curvature up to eps^-1 where a row is nearly 0 (width 1)
        assert abs(got - want) <= 1e-5 * (np.abs(dy).sum() * (1.0 + np.abs(direction).max())), (name, got, want)


def test_bounds_hold_for_an_fp32_evaluation(rng):
    """The stated bounds cover a plain fp32 evaluation with the stated roundings."""
    import torch
    bf = lambda a: torch.from_numpy(np.asarray(a, np.float64)).to(torch.bfloat16)  # noqa: E731
    n = 96
    q, k, v, g = (bf(rng.standard_normal((n, 128))) for _ in range(4))
    d = lambda t: t.double().numpy()  # noqa: E731
    o, lse = O.attention_forward(d(q), d(k), d(v))
    o, lse = bf(o), torch.from_numpy(lse).float()
    ref, bound = O.attention_backward(d(q), d(k), d(v), d(o), d(g), d(lse))
    qf, kf, vf, of, gf = (t.float() for t in (q, k, v, o, g))
    p = torch.exp(qf @ kf.T / O.SQRT_D - lse[:, None])
    ds = (p * (gf @ vf.T - (gf * of).sum(1, keepdim=True))).bfloat16().float()
    got = {"dq": (ds @ kf / O.SQRT_D).bfloat16(), "dk": (ds.T @ qf / O.SQRT_D).bfloat16(),
           "dv": (p.bfloat16().float().T @ gf).bfloat16()}
    for name in got:
        e = np.abs(d(got[name]) - ref[name])
        assert (e <= bound[name]).all(), name
        assert bound[name].mean() < 0.05 * np.abs(ref[name]).mean() + 0.05
