"""The ramped ("yarn") stretch of the frequencies pinned by counting turns instead of by its logarithms (Peng, Quesnelle,
Fan, Shippole: YaRN, 2023): a pair that makes beta_fast turns or more over the original context keeps its frequency,
one that makes beta_slow or fewer has it divided, and between the last of the former and the first of the latter the
share that is divided grows by equal steps from pair to pair. The oracle and the library's host code alike. No GPU."""
import math

import numpy as np
import pytest

import speculative_verify_paged_gb300 as sv
from oracle import rope

CASES = [   # r, theta, factor, beta_fast, beta_slow, original length
    (64, 10000.0, 40.0, 32.0, 1.0, 4096), (128, 10000.0, 16.0, 32.0, 1.0, 4096), (128, 500000.0, 4.0, 32.0, 1.0, 8192),
    (128, 1e6, 4.0, 32.0, 1.0, 32768), (96, 10000.0, 32.0, 20.0, 2.0, 2048), (20, 10000.0, 8.0, 32.0, 1.0, 4096), (64, 10000.0, 0.5, 32.0, 1.0, 4096),
    (128, 10000.0, 8.0, 4.0, 0.25, 1000), (6, 100.0, 2.0, 50.0, 3.0, 300), (64, 10000.0, 8.0, 32.0, 1e-4, 4096), (64, 10000.0, 8.0, 1e5, 1.0, 4096),
]


def by_turns(r, theta, factor, fast, slow, length):
    """The frequencies, from the turns that pair i = 0, 1, .. makes over the context (counted on past the last pair, to r - 1)."""
    turns = [length * theta ** (-2.0 * i / r) / (2 * math.pi) for i in range(r)]
    lo = max([i for i in range(r) if turns[i] >= fast], default=0)
    hi = min([i for i in range(r) if turns[i] <= slow], default=r - 1)
    out = []
    for i in range(r // 2):
        share = 0.0 if i <= lo else 1.0 if i >= hi else (i - lo) / (hi - lo)   # divided
        w = theta ** (-2.0 * i / r)
        out.append((1 - share) * w + share * (w / factor))
    return np.array(out), lo, hi


@pytest.fixture(scope="module", autouse=True)
def lib():
    sv.build()


@pytest.mark.parametrize("case", CASES)
def test_frequencies_by_counted_turns(case):
    r, theta, factor, fast, slow, length = case
    want, lo, hi = by_turns(*case)
    assert lo < hi
    w = rope.frequencies(r, theta)
    got, _ = rope.yarn(w, theta, factor, fast, slow, length)
    assert np.allclose(got, want, rtol=1e-12)
    s = {"kind": "yarn", "factor": factor, "beta_fast": fast, "beta_slow": slow, "original_length": length}
    assert np.allclose(sv.Rope(r, theta, scaling=s).inv_freq, want, rtol=1e-12)
    # kept, divided, and the steps between
    ratio = got / w
    assert np.allclose(ratio[:lo + 1], 1, rtol=1e-12) and np.allclose(ratio[hi:], 1 / factor, rtol=1e-12)
    steps = np.diff(ratio[lo:hi + 1])
    assert len(steps) == 0 or np.allclose(steps, (1 / factor - 1) / (hi - lo), rtol=1e-9)


def test_numbers_worked_out_by_hand():
    # 4096 / (2 pi) = 651.9 turns of pair 0, divided by 10000^(1/32) = 1.3335 from pair to pair: pair 10 makes 36.66, pair 11
    # 27.49 (32 lies between), pair 22 1.159, pair 23 0.869 (1 lies between); 13 steps of 1/13 from 10 to 23
    want, lo, hi = by_turns(64, 10000.0, 40.0, 32.0, 1.0, 4096)
    assert (lo, hi) == (10, 23)
    w = rope.frequencies(64)
    got, m = rope.yarn(w, 10000.0, 40.0, 32.0, 1.0, 4096)
    assert math.isclose(got[10], w[10], rel_tol=1e-12) and math.isclose(got[23], w[23] / 40, rel_tol=1e-12)
    assert math.isclose(got[16], w[16] * (7 / 13 + 6 / 13 / 40), rel_tol=1e-12)
    assert math.isclose(m, 1.3688879454113936, rel_tol=1e-12)   # 1 + ln(40) / 10, ln 40 = 3.688879454113936


def test_the_factor_on_cosine_and_sine():
    w = rope.frequencies(64)
    for factor, m in ((math.e, 1.1), (math.e ** 5, 1.5), (1.0, 1.0), (0.25, 1.0)):
        assert math.isclose(rope.yarn(w, 10000.0, factor, 32.0, 1.0, 4096)[1], m, rel_tol=1e-12)
        s = {"kind": "yarn", "factor": factor, "original_length": 4096}
        assert math.isclose(sv.Rope(64, scaling=s).scale, m, rel_tol=1e-6)   # (held in f32)
