"""The sines and cosines that h3_rope turns by: fp32 rows of pairs (1, 0) come
back as (cosine, sine) unchanged, since the products with 0 and 1 are exact."""
import numpy as np
import pytest
import torch

import audio_video_flow_gb300 as h3
from oracle import h3_train_oracle as O

pytestmark = pytest.mark.gpu


def turned_units(pos, axes, freqs, layout, backward, **kw):
    """[rows][axes freqs] cosines and sines of the call."""
    pairs = axes * freqs
    width = (2 * pairs + 3) // 4 * 4
    x = torch.zeros(len(pos), 1, width, device="cuda")
    first = slice(0, pairs) if layout == "half" else slice(0, 2 * pairs, 2)
    second = slice(pairs, 2 * pairs) if layout == "half" else slice(1, 2 * pairs, 2)
    x[..., first] = 1.0
    cfg = h3.make_rope_config(width, axes, freqs, dtype=h3.H3_FP32,
                              layout=h3.H3_ROPE_HALF if layout == "half" else h3.H3_ROPE_INTERLEAVED, **kw)
    out = torch.empty_like(x)
    h3.h3_rope(cfg, len(pos), torch.from_numpy(pos).cuda(), int(backward), x, out, 1, None, None, 0, width, width, width,
               width)
    torch.cuda.synchronize()
    assert h3.h3_sync_check(timeout_ms=60000) == 0
    y = out[:, 0].double().cpu().numpy()
    return y[:, first], y[:, second]


def check(pos, axes, freqs, layout="half", backward=False, **kw):
    """An angle within 2^-28 of a turn moves sine and cosine by at most 2 pi
    2^-28.  The functions are within 1 ulp of fp32 (a relative 2^-23), and
    bringing in the angle's last bits rounds once more (2^-24): 2^-22 covers
    both."""
    cos, sin = turned_units(pos, axes, freqs, layout, backward, **kw)
    turns = pos.astype(np.longdouble)[:, :, None] * (O.rope_frequencies(axes, freqs, theta=kw.get("theta", 10000.0)) / O.TWO_PI)
    angle = ((turns - np.round(turns)) * O.TWO_PI).reshape(len(pos), -1)
    for got, want, what in ((cos, np.cos(angle), "cosine"), (sin, (-1 if backward else 1) * np.sin(angle), "sine")):
        bound = 2 * np.pi * 2.0 ** -28 + 2.0 ** -22 * np.abs(want)
        worst = (np.abs(got - want) / bound).max()
        assert worst <= 1.0, f"{what}: {worst:.3g} times its bound"


@pytest.mark.parametrize("layout, freqs", [("half", 64), ("interleaved", 64), ("half", 13), ("interleaved", 13)])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("far", [1 << 10, 1 << 20, (1 << 31) - 1])
def test_angles(layout, freqs, backward, far):
    pos = np.random.default_rng(far + freqs).integers(-far, far, (4096, 1)).astype(np.int32)
    check(pos, 1, freqs, layout, backward)


@pytest.mark.parametrize("theta", [2.0 ** 40, 1e20, 3.4028234e38])
def test_angles_of_large_bases(theta):
    pos = np.random.default_rng(7).integers(-2 ** 31, 2 ** 31, (512, 2)).astype(np.int32)
    pos[:4] = [[2 ** 31 - 1, -2 ** 31], [-2 ** 31, 2 ** 31 - 1], [0, 1], [-1, 0]]
    check(pos, 2, 64, theta=float(np.float32(theta)))


def test_positions_next_to_quarter_turns():
    """Positions chosen among many so that the angle of the first frequency (one
    radian a position) lies nearest to a quarter, half or whole turn, or nearest
    to the middle between two of them."""
    p = np.arange(-(1 << 21), 1 << 21)
    eighths = (p.astype(np.longdouble) / O.TWO_PI * 8) % 1
    near = np.argsort(np.minimum(eighths, 1 - eighths))[:2000]
    check(p[near].astype(np.int32)[:, None], 1, 2)


def test_position_zero_changes_nothing():
    cos, sin = turned_units(np.zeros((3, 2), np.int32), 2, 8, "half", False)
    assert (cos == 1.0).all() and (sin == 0.0).all()
