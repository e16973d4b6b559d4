"""The angle of rotary positions at far positions and large frequencies, against exact arithmetic.

Bounds. The angle: 2^-64 turns a position in the fraction, 2^-33 at 32-bit positions; cut to 32
bits, 2^-32; rounded to f32 as half turns within +-1, 2^-26 turns: 2^-25.9 turns in all, 2^-23.2
radians, which moves a rotated (1, 0) by as much. Cosine and sine: 2 units in the last place of
f32, 2^-22 of 1 at most. So 2^-21.4 a component. The roundings are of either sign: over 4096
positions in a row the angle's mean error is that of the fraction, with 2^-22 / sqrt(4096) = 2^-28
of the roundings, and 2^-30.3 radians of the cut: below 2^-27 together.
"""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
getcontext().prec = 60


def _atan(n):
    """atan(1 / n) by its series."""
    t = s = Decimal(1) / n
    k = 1
    while abs(t) > Decimal(10) ** -58:
        t = -t / (n * n)
        k += 2
        s += t / k
    return s


TURN = 8 * (4 * _atan(5) - _atan(239))   # 2 pi, by Machin's formula


def angles(w, positions):
    """position * w modulo 2 pi, exact to far below a double."""
    return np.array([float((Decimal(int(p)) * Decimal(w)) % TURN) for p in positions])


def turned(lib, w, positions):
    """(cos, sin) that the kernel turns (1, 0) into, for one pair of frequency w, as doubles [n]."""
    n = len(positions)
    q = torch.zeros((1, n, 1, 2), device=DEV)
    q[..., 0] = 1.0
    pos = torch.tensor(np.asarray(positions, dtype=np.int64), dtype=torch.int32, device=DEV)[None]
    out, _ = lib.spec_rope(q, None, lib.Rope(2, inv_freq=[w]), positions=pos)
    c, s = out[0, :, 0].double().cpu().numpy().T
    return c, s


FAR = [0, 1, -1, 777, 131071, 16777217, 999999937, 2 ** 31 - 1, -2 ** 31, -2 ** 30 - 1]


@pytest.mark.parametrize("w", [1.0, 0.7498942093324559, 1e-5, 6.283185307179586, 7.5, -0.3, 100.25, 12345.678, 1e6 + 0.1, -3.7e8, 1e10 + 0.37,
                               2.0 ** 40 - 0.5])
def test_far_positions_of_any_frequency(lib, w):
    c, s = turned(lib, w, FAR)
    a = angles(w, FAR)
    assert np.abs(c - np.cos(a)).max() <= 2.0 ** -21.4 and np.abs(s - np.sin(a)).max() <= 2.0 ** -21.4


@pytest.mark.parametrize("start", [2 ** 31 - 4096, -2 ** 31, 2 ** 30, 100000])
@pytest.mark.parametrize("w", [1.0, 0.7498942093324559, 0.1, 3.0, 50.5])
def test_the_angle_is_not_off_on_average(lib, w, start):
    positions = np.arange(start, start + 4096)
    c, s = turned(lib, w, positions)
    a = angles(w, positions)
    err = s * np.cos(a) - c * np.sin(a)   # the sine of the difference
    assert np.abs(err).max() <= 2.0 ** -21 and abs(err.mean()) <= 2.0 ** -27
