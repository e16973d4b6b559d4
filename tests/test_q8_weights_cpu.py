"""How the 8-bit verify attention cuts an f16 weight into three e5m2 terms, over every weight
there is: bit by bit as the kernel does it, against the bounds that its header states. No GPU."""
import re

import numpy as np
import pytest
import torch

from test_launch_rules_cpu import source

SRC = source("attn_q8.cu")
TOP, MOVE = (float(re.search(r"%s = ([0-9.]+)f" % n, SRC).group(1)) for n in ("kTop", "kMove"))
CUT = float(re.search(r"kCut = ([0-9.]+)f", SRC).group(1))


def val(bits):
    return bits.astype(np.uint16).view(np.float16).astype(np.float64)


def bits(x):
    return x.astype(np.float16).view(np.uint16)


def e5m2(byte):
    return torch.from_numpy(byte.astype(np.uint8)).view(torch.float8_e5m2).double().numpy()


def near(h):
    return ((h.astype(np.uint32) + 0x80) & 0xff00).astype(np.uint16)


def weights():
    """Every f16 from 0 to what a weight of 2^kMove rounds to."""
    last = int(bits(np.array([2.0 ** MOVE]))[0])
    return np.arange(last + 1, dtype=np.uint16)


def cut(h):
    a = near(h)
    r = bits(val(h) - val(a))
    assert np.array_equal(val(r), val(h) - val(a))   # what is left is exact in f16
    b = near(r)
    s = bits(val(r) - val(b))
    assert np.array_equal(val(s), val(r) - val(b))
    t = bits(val(s) / CUT)
    assert np.array_equal(val(t), val(s) / CUT)
    terms = [e5m2(x >> 8) for x in (a, b, near(t))]
    assert all(np.isfinite(x).all() for x in terms)
    return terms[0] + terms[1] + CUT * terms[2]


def test_the_source_is_what_this_file_restates():
    body = SRC[SRC.index("void cut_weights"):SRC.index("__global__")]
    assert body.count("+ 0x00800080u") == 2 and body.count("& 0xFF00FF00u") == 1 and body.count("__byte_perm") == 3
    assert body.count("near(") == 4 and "__float2half2_rn(32.f)" in body and CUT == 1 / 32


def test_weights_are_their_terms():
    h = weights()
    x, y = val(h), cut(h)
    assert 2.0 ** 15.5 < x[-1] < 61440     # (from 61440 on the nearest first term would be an infinity)
    big = x >= 2.0 ** (TOP - 15)
    assert np.array_equal(x[big], y[big])   # f16's own rounding, 2^-11 relative, is all there is
    # below: 2^-21 of the terms and half a step of f16's subnormals, 2^-25
    assert np.abs(x - y)[~big].max() <= 2.0 ** -21 and 2.0 ** -21 + 2.0 ** -25 <= 2.0 ** (TOP - 25)


def test_the_terms_lean_to_neither_side():
    h = weights()[1:]
    x, y = val(h), cut(h)
    assert abs(((y - x) / x)[x >= 2.0 ** -14].mean()) < 2.0 ** -18


@pytest.mark.parametrize("h", [0x7fff])
def test_nan_becomes_zeros(h):
    # (NaN as conversions and subtractions give it; its row's sum holds the NaN)
    assert e5m2(near(np.array([h], np.uint16)) >> 8)[0] == 0
