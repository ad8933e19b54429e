"""Angles of the rotation at any frequency and position, against exact rational arithmetic.

Tolerance: as in the tests of gdr_qk_norm_rope (32 x 2^-24 of the magnitudes an output is formed from: 30
roundings; the angle's 2^-31 turn, 3e-9 rad, is a twentieth of one)."""
import math
from fractions import Fraction

import pytest
import torch

from gated_deltanet_rule_gb300 import gdr

pytestmark = pytest.mark.gpu

PI = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816, 10 ** 69)
FREQS = [1.0, 1e-6, 3.0, math.pi, 3.9999, 4.0, 10.0, -100.0, 1000.0, 1e6, -1.2345e9, 2.0 ** 40 + 1 / 3, 1e15, 2.0 ** 61, -(2.0 ** 62 - 2.0 ** 9), 5e-324]
POS = [0, 1, -1, 12345, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1, 1999999973]


def _exact(f, pos):
    turns = Fraction(f) * pos / (2 * PI)
    a = 2 * math.pi * float(turns - math.floor(turns))
    return math.cos(a), math.sin(a)


def _case(freqs, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(1, len(POS), 2, 64, generator=g)
    pos = torch.tensor([POS], dtype=torch.int64).int()
    w = torch.ones(64)
    return x, w, torch.tensor(freqs, dtype=torch.float64), pos


def _run(x, w, inv, pos, interleaved):
    d = [t.cuda() for t in (x, x, w, w, inv, pos)]
    out, _ = gdr.gdr_qk_norm_rope(*d, interleaved=interleaved)
    gdr.gdr_sync_status()
    return out.cpu().double()


@pytest.mark.parametrize("interleaved", [False, True])
def test_any_frequency(interleaved):
    x, w, inv, pos = _case(FREQS)
    out = _run(x, w, inv, pos, interleaved)
    y = x.double() / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-6)
    H = len(FREQS)
    for t, p in enumerate(POS):
        for j, f in enumerate(FREQS):
            lo, hi = (2 * j, 2 * j + 1) if interleaved else (j, j + H)
            c, s = _exact(f, p)
            a, b = y[0, t, :, lo], y[0, t, :, hi]
            tol = 32 * 2.0 ** -24 * (a.abs() + b.abs())
            for got, want in ((out[0, t, :, lo], a * c - b * s), (out[0, t, :, hi], b * c + a * s)):
                assert ((got - want).abs() <= tol).all(), (f, p, got, want)
    assert (out[..., 2 * H:] - y[..., 2 * H:]).abs().max() < 1e-5


@pytest.mark.parametrize("interleaved", [False, True])
def test_no_angle_is_nan(interleaved):
    """A frequency that is infinite, nan or past 2^62 has no angle: its pair is nan, the others are as without it."""
    bad = {1: math.inf, 3: -math.inf, 4: math.nan, 6: 2.0 ** 62, 7: -1e300}
    good = [1.0 / (j + 1) for j in range(8)]
    x, w, inv, pos = _case(good)
    want = _run(x, w, inv, pos, interleaved)
    for j, f in bad.items():
        inv[j] = f
    out = _run(x, w, inv, pos, interleaved)
    hit = torch.zeros(64, dtype=torch.bool)
    for j in bad:
        hit[list((2 * j, 2 * j + 1) if interleaved else (j, j + 8))] = True
    assert torch.isnan(out[..., hit]).all() and torch.equal(out[..., ~hit], want[..., ~hit])
