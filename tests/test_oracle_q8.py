"""The 8-bit oracle against things other than itself: pages by hand, the
rounding by brute force, a straightforward dense model."""
import numpy as np
import pytest
import torch

from oracle import fp8
from oracle import q8


def test_exponent_by_hand():
    for A, e in ((448.0, 0), (448.0 + 2.0 ** -14, 1), (224.0, -1), (225.0, 0), (1.75, -8), (1.7500001, -7), (1.0, -8), (0.0, -32),
                 (1e-30, -32), (3e38, 32), (np.inf, 32), (448 * 2.0 ** 32, 32), (448 * 2.0 ** -32, -32)):
        assert q8.exponent(A) == e, A


def test_page_by_hand():
    assert q8.page_bytes(8, 128, 16) == 8 * 2048 + 128 and q8.page_bytes(1, 128, 16) == 2048 + 128
    assert q8.page_bytes(32, 128, 16) == 32 * 2048 + 128 and q8.page_bytes(33, 64, 8) == 33 * 512 + 256
    c = np.zeros((1, 2, 16, 128), np.uint8)
    c[0, 1, 5, 70] = 9
    pool = q8.join(c, np.array([[2.0, 0.5]], np.float32))
    assert pool[0, 2048 + 5 * 128 + 70] == 9 and pool[0, :4096].sum() == 9
    assert pool[0, 4096:4104].tobytes() == np.array([2.0, 0.5], np.float32).tobytes() and not pool[0, 4104:].any()
    codes, scales = q8.split(pool, 2, 128, 16)
    assert np.array_equal(codes, c) and scales.tolist() == [[2.0, 0.5]]


def test_codes_are_the_nearest():
    x = torch.randn(4000, generator=torch.Generator().manual_seed(0)).numpy() * np.exp2(np.arange(4000) % 40 - 30)
    x = x.astype(np.float32)
    scale = 2.0 ** q8.exponent(float(np.abs(x).max()))
    v = fp8.decode(q8.encode(x, scale)) * scale
    grid = fp8.code_values()
    grid = grid[np.isfinite(grid)] * scale
    assert (np.abs(v - x) <= np.abs(grid[None] - x[:, None]).min(1)).all()
    assert np.abs(x).max() <= 448 * scale and np.abs(x).max() > 224 * scale
    assert q8.encode(np.float32([np.nan, np.inf, -np.inf]), 1.0).tolist() == [0, 0x7E, 0xFE]


@pytest.mark.parametrize("n", [1, 5, 16, 37])
def test_append_against_a_dense_model(n):
    # rows that arrive in pieces, later ones larger: a block's scale grows, and its rows stay within a rounding of the
    # final scale of what they were
    rng = np.random.default_rng(n)
    H, d, bs, rounds = 2, 32, 16, 5
    k = v = np.zeros((20, q8.page_bytes(H, d, bs)), np.uint8)
    table = rng.permutation(20)[None, :19]
    rows, L = [], 0
    for i in range(rounds):
        x = (rng.standard_normal((1, n, H, d)) * 3.0 ** i).astype(np.float32)
        rows.append(x[0])
        L += n
        if L > 19 * bs:
            break
        k, v = q8.append(k, v, x, -x, table, [L], bs)
    rows = np.concatenate(rows)
    got = q8.dense(k, table[0], L, H, d, bs)
    assert np.array_equal(q8.dense(v, table[0], L, H, d, bs), -got)
    _, scales = q8.split(k[table[0]], H, d, bs)
    s = np.repeat(scales, bs, axis=0)[:L].astype(float)
    for page in range((L + bs - 1) // bs):   # the smallest power of two that holds the block (the first rows' growth only adds)
        top = np.abs(rows[page * bs:(page + 1) * bs]).max(axis=(0, 2))
        for g in range(H):
            assert scales[page, g] == 2.0 ** q8.exponent(float(top[g]))
    # two roundings at most: relative 2^-4 each above the subnormals, half a step of 2^-9 s below, at every scale so far
    err = np.abs(got - rows)
    assert (err <= 2.2 * np.maximum(2.0 ** -4 * np.abs(rows), 2.0 ** -10 * s[..., None])).all()


def test_append_moves_codes_exactly_but_for_subnormals():
    # a block with scale 2^-8 whose new row needs 2^-3: codes down five binades
    H, d, bs = 1, 16, 16
    k = np.zeros((1, q8.page_bytes(H, d, bs)), np.uint8)
    first = np.full((1, 1, H, d), 1.5, np.float32)
    first[..., 0] = 2.0 ** -10
    first[..., 1] = 1.625
    first[..., 2] = 2.0 ** -14
    k1, _ = q8.append(k, k, first, first, [[0]], [1], bs)
    k2, _ = q8.append(k1, k1, first * 0 + 32.0, first, [[0]], [2], bs)
    c1, s1 = q8.split(k1, H, d, bs)
    c2, s2 = q8.split(k2, H, d, bs)
    assert s1[0, 0] == 2.0 ** -8 and s2[0, 0] == 2.0 ** -3
    v = q8.values(c2, s2)
    # 1.5 / 2^-3 = 12 is normal, 2^-10 four steps of the subnormals, 2^-9 * 2^-3; 2^-14 lies below half a step
    assert (v[0, 0, 0] == np.r_[2.0 ** -10, 1.625, 0.0, np.full(13, 1.5)]).all()
    assert q8.values(c1, s1)[0, 0, 0, 2] == 2.0 ** -14
    assert (v[0, 0, 1] == 32.0).all()


def test_reading_takes_any_scale():
    c = np.full((1, 1, 1, 4), 0x38, np.uint8)   # the code of 1
    for s, want in ((0.0, q8.LO), (np.nan, q8.LO), (-1.0, q8.LO), (np.inf, q8.HI), (0.3, float(np.float32(0.3)))):
        assert (q8.values(c, np.array([[s]], np.float32)) == want).all()
