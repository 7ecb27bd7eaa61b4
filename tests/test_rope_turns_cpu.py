"""The frequency table of h3_rope on the host: turns per position in 64-bit
fixed point against 80-digit arithmetic on the configuration's own numbers."""
import ctypes
import os
import subprocess
from decimal import Decimal, getcontext

import numpy as np
import pytest

import audio_video_flow_gb300 as h3
from audio_video_flow_gb300 import _build

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211707")
SCALINGS = {"none": h3.H3_ROPE_SCALE_NONE, "linear": h3.H3_ROPE_SCALE_LINEAR, "ntk": h3.H3_ROPE_SCALE_NTK,
            "yarn": h3.H3_ROPE_SCALE_YARN}
# Units of 2^-64 turns.  The series is held in 128-bit mantissas: each of at
# most 128 steps and the root's Newton step are relative errors below 2^-90 of
# numbers below 2^62 units, so below a unit in all, and the result is rounded to
# a whole one.  At position 2^31 that is 2^-32 of a turn.
UNITS = 2


@pytest.fixture(scope="module")
def turns(tmp_path_factory):
    d = tmp_path_factory.mktemp("turns")
    (d / "t.cpp").write_text('#include "rope_turns.h"\n'
                             'extern "C" void turns(const h3_rope_config* c, uint64_t* t) { h3::rope_turns(*c, t); }\n')
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build._nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-o", str(d / "t.so"),
                    str(d / "t.cpp"), "-I", os.path.dirname(h3.HEADER), "-I", _build.CSRC, "-I", cuda], check=True)
    f = ctypes.CDLL(str(d / "t.so")).turns
    f.argtypes = [ctypes.POINTER(h3.RopeConfig), ctypes.POINTER(ctypes.c_uint64)]

    def table(cfg):
        out = (ctypes.c_uint64 * (cfg.n_axes * cfg.n_freqs))()
        f(ctypes.byref(cfg), out)
        return [list(out[a * cfg.n_freqs:(a + 1) * cfg.n_freqs]) for a in range(cfg.n_axes)]
    return table


def exact(cfg, scaling, axis):
    """The definition, in units of 2^-64 turns."""
    getcontext().prec = 80
    F, theta, s = cfg.n_freqs, Decimal(cfg.theta), Decimal(cfg.factor)   # the fp32 values, exactly
    scaled = scaling != "none" and (cfg.scaled_axes >> axis) & 1
    out = []
    for f in range(F):
        w = (theta.ln() * -f / F).exp()
        if scaled and scaling == "linear":
            w /= s
        elif scaled and scaling == "ntk":
            w = ((theta.ln() + s.ln() * F / (F - 1)) * -f / F).exp()
        elif scaled and scaling == "yarn":
            n = Decimal(cfg.trained_length) * w / (2 * PI)
            g = min(max((n - Decimal(cfg.alpha)) / (Decimal(cfg.beta) - Decimal(cfg.alpha)), Decimal(0)), Decimal(1))
            w = g * w + (1 - g) * w / s
        out.append(w / (2 * PI) * 2 ** 64)
    return out


def check(turns, scaling, **kw):
    cfg = h3.make_rope_config(256, scaling=SCALINGS[scaling], **kw)
    table = turns(cfg)
    for a in range(cfg.n_axes):
        for f, want in enumerate(exact(cfg, scaling, a)):
            assert abs(Decimal(table[a][f]) - want) <= UNITS, (scaling, kw, a, f)


# bases from next to 1 to the largest fp32, on both sides of 2^40
THETAS = [float(np.nextafter(np.float32(1), np.float32(2))), 1.5, 2.0, 100.0, 10000.0, 500000.0, 1e9, 2.0 ** 40 * 0.999,
          2.0 ** 40, 1e13, 1e20, 1e38, 3.4028234e38]


@pytest.mark.parametrize("scaling", sorted(SCALINGS))
@pytest.mark.parametrize("theta", THETAS)
def test_bases(turns, scaling, theta):
    for n_freqs in (2, 3, 16, 43, 64, 127, 128):
        check(turns, scaling, n_axes=1, n_freqs=n_freqs, theta=theta, factor=8.0, trained_length=4096.0)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn"])
@pytest.mark.parametrize("factor", [1.0, float(np.nextafter(np.float32(1), np.float32(2))), 1.5, 3.0, 32.0, 1e6, 1e13,
                                    3.4028234e38])
def test_factors(turns, scaling, factor):
    for n_freqs in (2, 32, 64):
        check(turns, scaling, n_axes=1, n_freqs=n_freqs, factor=factor, trained_length=4096.0)


@pytest.mark.parametrize("trained, alpha, beta", [
    (4096.0, 1.0, 32.0), (4096.0, 0.0, 1e-3), (1.0, 0.0, 0.125), (131072.0, 31.999, 32.0), (1e30, 1e25, 1.5e25),
    (4096.0, 0.5, float(np.nextafter(np.float32(0.5), np.float32(1)))), (3.4e38, 0.0, 3.4e38), (1.0, 1e-38, 1.0)])
def test_ramps(turns, trained, alpha, beta):
    """Ramps over many frequencies, over few, and next to a step."""
    for theta in (10000.0, 1e13):
        for n_freqs in (1, 64, 128):
            check(turns, "yarn", n_axes=1, n_freqs=n_freqs, theta=theta, factor=40.0, trained_length=trained, alpha=alpha,
                  beta=beta)


def test_a_frequency_on_the_ramp(turns):
    """The ramp put round each frequency in turn, as narrow as fp32 allows and wider."""
    for f in range(0, 64, 7):
        n = np.float32(4096 * 10000.0 ** (-f / 64) / (2 * np.pi))
        for width in (0, 1, 100):
            lo = n
            hi = np.nextafter(n, np.float32(np.inf))
            for _ in range(width):
                lo, hi = np.nextafter(lo, np.float32(0)), np.nextafter(hi, np.float32(np.inf))
            check(turns, "yarn", n_axes=1, n_freqs=64, factor=40.0, trained_length=4096.0, alpha=float(lo), beta=float(hi))


@pytest.mark.parametrize("scaled_axes", range(8))
def test_axes(turns, scaled_axes):
    for scaling in ("linear", "ntk", "yarn"):
        check(turns, scaling, n_axes=3, n_freqs=16, factor=4.0, trained_length=512.0, scaled_axes=scaled_axes)
