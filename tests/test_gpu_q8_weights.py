"""The weights of verify attention over 8-bit block-scaled pools, seen through its outputs.

Bounds. Values are of one sign, so an output's relative error is at most its weights': half a
step of f16, 2^-11 (all weights here lie within 2^-15 of the row's largest), and what the
scores bring: q and the keys' codes are exact in their terms, so 2^-22 of the power of two and
2^-24 of scores up to 2^4, below 2^-19 in all. Then half a step of bf16 at the output, where it
lies: 2^-8 for outputs in [1, 2). (A weight cut into three e5m2 terms by truncation is up to
2^-9.2 too large, which this bound shows.)
"""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import q8 as oq8

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, L = 48, 1000


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def pools(lib, first, seed):
    """Keys that are zero but for dim 0 (`first`, [L]), values in [1, 2) with one scale: pools, table, and the values."""
    g = torch.Generator().manual_seed(seed)
    K = torch.zeros((B, L, 1, 128))
    K[..., 0, 0] = first
    V = 1.0 + torch.randint(0, 8, (B, L, 1, 128), generator=g) / 8.0
    V[..., 0] = 1.875
    nb = -(-L // 16)
    kc, vc = lib.alloc_q8_pools(B * nb, 1, 128)
    table = torch.arange(B * nb, dtype=torch.int32).reshape(B, nb).to(DEV)
    lib.kv_block_append_q8(K.to(DEV), V.to(DEV), kc, vc, table, i32([L] * B))
    for b in (0, B - 1):   # (nothing is rounded on the way in)
        for pool, x in ((kc, K), (vc, V)):
            assert np.array_equal(oq8.dense(pool.cpu().numpy(), table[b].cpu().numpy(), L, 1, 128), x[b].double().numpy())
    return kc, vc, table, K, V


def errors(out, q, K, V, scale):
    got = out.double().cpu().numpy()
    n = q.shape[1]
    ref = np.stack([oatt.dense_attention(q[b].double().numpy(), K[b].double().numpy(), V[b].double().numpy(), n, scale) for b in range(B)])
    assert (ref >= 1).all() and (ref < 2).all()
    return got - ref, ref


ROWS = [(4, 1), (8, 1), (12, 1), (8, 4), (8, 5), (8, 6), (8, 8), (16, 7)]


@pytest.mark.parametrize("H_q,n", ROWS)
@pytest.mark.parametrize("mantissa", [0x092, 0x0c9, 0x1ff, 0x2aa, 0x3ff])
def test_one_weight_over_and_over(lib, H_q, n, mantissa):
    # one key's weight is 2^5, all others' are 1 + mantissa / 2^10, exactly an f16
    w = 1 + mantissa / 1024
    first = torch.zeros(L)
    first[0] = 448.0
    scale = (5 - math.log2(w)) * math.log(2) / 448
    kc, vc, table, K, V = pools(lib, first, mantissa)
    q = torch.zeros((B, n, H_q, 128))
    q[..., 0] = 1.0
    out = lib.spec_verify_attn_q8(q.bfloat16().to(DEV), kc, vc, table, i32([L] * B), softmax_scale=scale)
    err, ref = errors(out, q, K, V, scale)
    assert np.abs(err).max() <= 2.0 ** -8 + 2.0 * (2.0 ** -11 + 2.0 ** -19)


@pytest.mark.parametrize("H_q,n", ROWS)
def test_weights_lean_to_neither_side(lib, H_q, n):
    # weights of every mantissa: the errors' mean over all outputs. bf16's roundings are even over +-2^-8, a deviation of
    # 2^-8.8; 48 x 127 outputs of other values make it 2^-15.1 for their mean. The weights' own roundings, 2^-11.8 each, add
    # less than 2^-15.8 over the some 300 keys that hold a row's weight. Together 2^-14.9, and four times that as the bound
    # (rows of other sizes only make the deviation smaller).
    g = torch.Generator().manual_seed(n)
    first = torch.randint(-14, 15, (L,), generator=g).float()
    kc, vc, table, K, V = pools(lib, first, 77)
    q = torch.zeros((B, n, H_q, 128))
    q[..., 0] = torch.randint(8, 16, (B, n, H_q), generator=g) / 8.0
    scale = 3.0 / 28
    out = lib.spec_verify_attn_q8(q.bfloat16().to(DEV), kc, vc, table, i32([L] * B), softmax_scale=scale)
    err, _ = errors(out, q, K, V, scale)
    assert np.abs(err).max() <= 2.0 ** -8 + 2.0 * (2.0 ** -11 + 2.0 ** -19)
    assert abs(err.mean()) <= 2.0 ** -12.9
