"""Oracle for rotary positions in fp64 ("KV Cache + Speculative Decoding",
section 6.3, _rope: consecutive pairs; the half layout pairs dim i with dim
i + r / 2), and the frequencies of the usual ways to stretch a context.
"""
import math

import numpy as np


def frequencies(r, theta=10000.0):
    return np.array([theta ** (-2.0 * i / r) for i in range(r // 2)])


def linear(w, factor):
    return w / factor


def llama3(w, factor, low, high, original_length):
    """Wavelengths above original_length / low divided by factor, below original_length / high kept, between
    them interpolated linearly in 1 / wavelength."""
    out = []
    for x in w:
        length = 2 * math.pi / x
        if length < original_length / high:
            out.append(x)
        elif length > original_length / low:
            out.append(x / factor)
        else:
            s = (original_length / length - low) / (high - low)
            out.append((1 - s) * x / factor + s * x)
    return np.array(out)


def yarn(w, theta, factor, beta_fast, beta_slow, original_length):
    """(frequencies, factor on cos and sin)."""
    r = 2 * len(w)

    def dim(turns):
        return r * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(theta))
    lo, hi = max(math.floor(dim(beta_fast)), 0), min(math.ceil(dim(beta_slow)), r - 1)
    if lo == hi:
        hi += 0.001
    ramp = np.clip((np.arange(len(w)) - lo) / (hi - lo), 0, 1)
    return w / factor * ramp + w * (1 - ramp), 0.1 * math.log(factor) + 1 if factor > 1 else 1.0


def rotate(x, positions, w, interleaved=False, offset=0, scale=1.0):
    """x [B, n, H, d] with dims offset .. offset + 2 len(w) - 1 turned by positions [B, n] * w, times scale."""
    x = np.array(x, dtype=np.float64)
    r = 2 * len(w)
    # the product position * w_i is exact to 2^-53 of itself: far below what any test here resolves
    a = np.asarray(positions, dtype=np.float64)[..., None, None] * w
    c, s = scale * np.cos(a), scale * np.sin(a)
    part = x[..., offset:offset + r]
    if interleaved:
        i, j = np.arange(0, r, 2), np.arange(1, r, 2)
    else:
        i, j = np.arange(r // 2), np.arange(r // 2, r)
    u, v = part[..., i].copy(), part[..., j].copy()
    part[..., i], part[..., j] = u * c - v * s, v * c + u * s
    return x
