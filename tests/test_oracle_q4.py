"""The 4-bit oracle against things other than itself: hand-packed records, the
rounding's definition by brute force, dense round trips and the window's mask
written out."""
import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import q4


def test_quantize_is_the_nearest_code():
    x = np.random.default_rng(0).standard_normal((50, 128)).astype(np.float32)
    c, s, m = q4.quantize(x)
    v = np.arange(16)[None, None] * s.astype(float)[:, None, None] + m.astype(float)[:, None, None]
    best = np.abs(v - x[..., None]).min(axis=-1)
    got = np.abs(q4.values(c, s, m) - x)
    assert (got <= best * (1 + 1e-5) + 1e-9).all()
    assert (got <= 0.51 * s.astype(float)[:, None] + 2.0 ** -10).all()   # half a step, and the minimum's own rounding


def test_quantize_special_rows():
    z = np.zeros((1, 64), np.float32)
    c, s, m = q4.quantize(z)
    assert (c == 0).all() and s[0] == np.float16(2.0 ** -24) and m[0] == 0
    c, s, m = q4.quantize(z + 3.5)
    assert (c == 0).all() and (q4.values(c, s, m) == 3.5).all()
    n = z.copy(); n[0, 0], n[0, 1] = np.nan, 15.0
    c, s, m = q4.quantize(n)
    assert c[0, 0] == 0 and c[0, 1] == 15 and (c[0, 2:] == 0).all()
    c, s, m = q4.quantize(z * np.nan)
    assert (q4.values(c, s, m) == 0).all()
    i = z.copy(); i[0, 0], i[0, 1] = np.inf, -np.inf
    c, s, m = q4.quantize(i)
    assert np.isfinite(q4.values(c, s, m)).all() and c[0, 0] == 15 and c[0, 1] == 0


def test_record_bytes_by_hand():
    # d = 128, 16 slots: slot 5, head dim 70 of K: chunk 70 // 32 = 2, stored at 2 ^ ((5 >> 1) & 3) = 0,
    # byte (70 // 2) % 16 = 3 of it, the low four bits (70 is even)
    c = np.zeros((16, 128), np.uint8); c[5, 70] = 9
    s = np.full(16, 2.0, np.float16); m = np.full(16, -1.0, np.float16)
    rec = q4.pack("k", c, s, m)
    assert rec.shape == (16 * 64 + 64,) and rec[5 * 64 + 0 * 16 + 3] == 9 and rec[:1024].sum() == 9
    assert bytes(rec[1024:1028]) == np.float16(2.0).tobytes() + np.float16(-1.0).tobytes()
    c = np.zeros((16, 128), np.uint8); c[5, 70] = 9
    rec = q4.pack("v", c, s, m)
    assert rec[70 * 8 + 2] == 9 << 4 and rec[:1024].astype(int).sum() == 9 << 4


@pytest.mark.parametrize("d,bs", [(128, 16), (64, 8), (256, 32), (96, 16)])
@pytest.mark.parametrize("kind", ["k", "v"])
def test_pack_and_unpack_are_inverse(kind, d, bs):
    rng = np.random.default_rng(d + bs)
    c = rng.integers(0, 16, (3, 2, bs, d)).astype(np.uint8)
    s, m = (rng.standard_normal((3, 2, bs)).astype(np.float16) for _ in range(2))
    c2, s2, m2 = q4.unpack(kind, q4.pack(kind, c, s, m), d, bs)
    assert np.array_equal(c, c2) and np.array_equal(s, s2) and np.array_equal(m, m2)


def test_append_then_dense_is_the_quantised_rows():
    rng = np.random.default_rng(4)
    bs, d, H = 16, 32, 2
    k, v = (rng.standard_normal((2, 21, H, d)).astype(np.float32) for _ in range(2))
    table, lens = np.array([[3, 1, -1], [0, 4, 2]]), np.array([25, 40])
    kc, vc = (rng.integers(0, 64, (5, H, bs * (d // 2 + 4))).astype(np.uint8) for _ in range(2))
    k2, v2 = q4.append(kc, vc, k, v, table, lens, bs)
    for kind, old, new, x in (("k", kc, k2, k), ("v", vc, v2, v)):
        for b, L in enumerate(lens):
            want = q4.dense(kind, old, table[b], L, d, bs)
            want[L - 21:] = q4.values(*q4.quantize(x[b]))
            assert np.array_equal(q4.dense(kind, new, table[b], L, d, bs), want)


@pytest.mark.parametrize("n,L,W,S", [(1, 1, 1, 0), (3, 20, 4, 0), (3, 20, 4, 2), (5, 9, 30, 3), (2, 12, 5, 11)])
def test_window_visibility_is_the_statement(n, L, W, S):
    t, p = np.arange(L)[None], np.arange(L - n, L)[:, None]
    want = (t <= p) & ((p - t < W) | (t < S))
    got = oatt.window_visibility(n, L, W, S)
    assert np.array_equal(got, want) and got.any(axis=1).all()
    if W >= L:
        assert np.array_equal(got, np.tril(np.ones((n, L), bool), L - n))


def test_masked_attention_is_attention_over_the_visible_keys():
    rng = np.random.default_rng(1)
    q, K, V = rng.standard_normal((1, 4, 8)), rng.standard_normal((30, 2, 8)), rng.standard_normal((30, 2, 8))
    vis = oatt.window_visibility(1, 30, 6, 3)
    K2, V2 = K.copy(), V.copy()
    K2[~vis[0]], V2[~vis[0]] = np.nan, np.inf
    got = oatt.dense_attention(q, K2, V2, 1, 0.3, visible=vis)
    keep = np.r_[0:3, 24:30]
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), torch.from_numpy(K[keep]).transpose(0, 1).repeat_interleave(2, 0),
        torch.from_numpy(V[keep]).transpose(0, 1).repeat_interleave(2, 0), scale=0.3).transpose(0, 1).numpy()
    assert np.allclose(got, want, atol=1e-12)
