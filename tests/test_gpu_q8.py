"""The 8-bit block-scaled paged cache on the GPU against the oracle: append
(bit-exact), read-back (exact), verify attention, and a run of them together
with rotary positions."""
import math

import numpy as np
import pytest
import torch

from oracle import q8 as oq8
from oracle import rope as orope
from q8_utils import check_q8_attention, q8_pools, q8_reference, table_for

pytestmark = pytest.mark.gpu
DEV = "cuda"


def status0():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ----------------------------------------------------------------- append ---

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,bs,H,n,lens", [
    (128, 16, 2, 1, (1, 16, 17, 300)), (128, 16, 8, 5, (5, 20, 21, 35)), (128, 16, 1, 37, (37, 50, 64)),
    (128, 16, 3, 200, (200, 333)), (64, 8, 2, 3, (3, 8, 30)), (96, 16, 2, 19, (19, 40)), (256, 32, 1, 70, (70, 101)),
    (16, 64, 2, 64, (64, 65, 100)), (144, 24, 1, 9, (9, 30)), (48, 1, 3, 4, (4, 9)), (256, 64, 1, 61, (61, 130)), (32, 7, 2, 10, (10, 33)),
])
def test_append_is_bit_exact(lib, dtype, d, bs, H, n, lens):
    table, total = table_for(lens, bs, seed=d + n, max_blocks=-(-max(lens) // bs) + 2)
    kc, vc = q8_pools(total, H, d, bs, seed=n)
    g = torch.Generator().manual_seed(7)
    k, v = (torch.randn((len(lens), n, H, d), generator=g) for _ in range(2))
    k *= torch.exp2(torch.randint(-12, 13, (len(lens), n, H, 1), generator=g).float())   # blocks that grow and blocks that do not
    v[1:] *= 1e-5
    k, v = k.to(dtype), v.to(dtype)
    k[0, 0, 0], v[0, 0, 0, :7] = 0.25, 100.0
    kd, vd = kc.to(DEV), vc.to(DEV)
    st = status0()
    lib.kv_block_append_q8(k.to(DEV), v.to(DEV), kd, vd, table.to(DEV), i32(lens), block_size=bs, status=st)
    want = oq8.append(kc.numpy(), vc.numpy(), k.float().numpy(), v.float().numpy(), table.numpy(), lens, bs)
    assert int(st) == 0
    for got, ref in zip((kd, vd), want):
        assert np.array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_token_after_token(lib, dtype):
    # a block filled by single tokens of growing and shrinking size: every growth moves the codes before it
    H, L = 2, 40
    kc, vc = lib.alloc_q8_pools(4, H, 128)
    ref = [kc.cpu().numpy(), vc.cpu().numpy()]
    table = i32([[2, 0, 3]])
    g = torch.Generator().manual_seed(5)
    for t in range(1, L + 1):
        k, v = (torch.randn((1, 1, H, 128), generator=g) * 2.0 ** int(torch.randint(-6, 7, (1,), generator=g)) for _ in range(2))
        k, v = k.to(dtype), v.to(dtype)
        lib.kv_block_append_q8(k.to(DEV), v.to(DEV), kc, vc, table, i32([t]))
        ref = oq8.append(*ref, k.float().numpy(), v.float().numpy(), table.cpu().numpy(), [t])
    assert np.array_equal(kc.cpu().numpy(), ref[0]) and np.array_equal(vc.cpu().numpy(), ref[1])


def test_append_special_values(lib):
    # NaN, infinities, zero, tiny and huge rows, a block of nothing but NaN, and one whose rows end at an edge of 448 * 2^e
    x = torch.randn((1, 128, 1, 128), generator=torch.Generator().manual_seed(1))
    x[0, 0:16] = 0.0
    x[0, 16:32] = float("nan")
    x[0, 33, 0, 5], x[0, 34, 0, 9] = float("nan"), float("inf")
    x[0, 50, 0, 0] = -float("inf")
    x[0, 64:80] = 3e38
    x[0, 80:96] *= 1e-30
    x[0, 96:112] = torch.linspace(-448, 448, 2048).view(16, 1, 128) * 2.0 ** -5
    x[0, 112:] = torch.linspace(-448, 448, 2048).view(16, 1, 128) * 1.001
    for dtype in (torch.float32, torch.bfloat16):
        y = x.to(dtype)
        table, lens = torch.tensor([[2, 0, 1, 5, 4, 3, 7, 6]], dtype=torch.int32), [128]
        kc, vc = q8_pools(8, 1, 128, 16, seed=3)
        kd, vd = kc.to(DEV), vc.to(DEV)
        lib.kv_block_append_q8(y.to(DEV), -y.to(DEV), kd, vd, table.to(DEV), i32(lens))
        want = oq8.append(kc.numpy(), vc.numpy(), y.float().numpy(), -y.float().numpy(), table.numpy(), lens)
        assert np.array_equal(kd.cpu().numpy(), want[0]) and np.array_equal(vd.cpu().numpy(), want[1])
        back, _ = lib.kv_block_gather_q8(kd, vd, table.to(DEV), i32(lens), i32([0]), 128, 128, out_dtype=torch.float32)
        assert torch.isfinite(back).all()


def test_append_over_scales_of_other_kinds(lib):
    # pages filled elsewhere: scales that are no powers of two, zero, negative, NaN or infinite; new rows behind them
    H, n, L = 8, 3, 10
    kc, vc = q8_pools(2, H, 128, 16, seed=4, spread=False)
    odd = torch.tensor([0.3, 1e-5, 0.0, -1.0, float("nan"), float("inf"), 3.7e7, 2.0 ** -40])
    for pool in (kc, vc):
        lib.q8_views(pool, H, 128)[1][:] = odd
    k, v = (torch.randn((1, n, H, 128), generator=torch.Generator().manual_seed(s)).bfloat16() for s in (1, 2))
    kd, vd = kc.to(DEV), vc.to(DEV)
    lib.kv_block_append_q8(k.to(DEV), v.to(DEV), kd, vd, i32([[1]]), i32([L]))
    want = oq8.append(kc.numpy(), vc.numpy(), k.float().numpy(), v.float().numpy(), [[1]], [L])
    for got, ref in zip((kd, vd), want):
        assert np.array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_at_any_element(lib, dtype):
    # new rows and read-back buffers that start at an odd element of their storage
    H, n, lens = 3, 21, [40, 21]
    table, total = table_for(lens, 16, seed=5)
    kc, vc = (p.to(DEV) for p in q8_pools(total, H, 128, 16, seed=5))
    k2, v2 = kc.clone(), vc.clone()
    size = 2 * n * H * 128
    flat = torch.randn(2 * size + 8, generator=torch.Generator().manual_seed(5)).to(dtype).to(DEV)
    k, v = (flat[o:o + size].view(2, n, H, 128) for o in (1, size + 3))
    lib.kv_block_append_q8(k, v, kc, vc, table.to(DEV), i32(lens))
    lib.kv_block_append_q8(k.clone(), v.clone(), k2, v2, table.to(DEV), i32(lens))
    assert torch.equal(kc, k2) and torch.equal(vc, v2)
    dst = torch.full((2 * size + 8,), 7.0, dtype=dtype, device=DEV)
    out = [dst[o:o + size].view(2, n, H, 128) for o in (1, size + 3)]
    start = i32([25, -4])
    lib.kv_block_gather_q8(kc, vc, table.to(DEV), i32(lens), start, n, 128, k_out=out[0], v_out=out[1])
    want = lib.kv_block_gather_q8(kc, vc, table.to(DEV), i32(lens), start, n, 128, out_dtype=dtype)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert (dst[[0, size + 1, size + 2] + list(range(2 * size + 3, 2 * size + 8))] == 7).all()


def test_append_bad_lengths_and_blocks_leave_the_pools(lib):
    table = torch.tensor([[0, 1], [99, 99], [2, 3], [4, -1]], dtype=torch.int32, device=DEV)
    kc, vc = (p.to(DEV) for p in q8_pools(6, 2, 128, 16, seed=5))
    k0, v0 = kc.clone(), vc.clone()
    new = torch.randn((4, 4, 2, 128), device=DEV)
    st = status0()
    # shorter than n_new; a block outside the pool; longer than the table; a block of -1
    lib.kv_block_append_q8(new, new, kc, vc, table, i32([3, 20, 33, 20]), status=st)
    assert int(st) == 1 | 2
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_strided_pages(lib):
    # pages of one layer inside a pool of [num_blocks][layers][page]
    H, nb, layers = 2, 7, 3
    page = lib.q8_page_bytes(H, 128)
    small = [torch.stack([q8_pools(nb, H, 128, 16, seed=10 * s + i)[0] for i in range(layers)], 1).to(DEV) for s in range(2)]
    big_k, big_v = small
    k0, v0 = big_k.clone(), big_v.clone()
    new = torch.randn((2, 20, H, 128), device=DEV).bfloat16()
    table, lens = i32([[1, 4, 6], [5, 0, 2]]), i32([25, 40])
    layout = (layers * page, 0, 0)
    kl, vl = big_k.view(-1)[page:], big_v.view(-1)[page:]
    lib.kv_block_append_q8(new, new, kl, vl, table, lens, layout=layout, num_blocks=nb)
    dense_k, dense_v = k0[:, 1].contiguous(), v0[:, 1].contiguous()
    lib.kv_block_append_q8(new, new, dense_k, dense_v, table, lens)
    k0[:, 1], v0[:, 1] = dense_k, dense_v
    assert torch.equal(big_k, k0) and torch.equal(big_v, v0)
    start = i32([3, 17])
    a = lib.kv_block_gather_q8(kl, vl, table, lens, start, 9, 128, layout=layout, num_blocks=nb, H_kv=H)
    b = lib.kv_block_gather_q8(dense_k, dense_v, table, lens, start, 9, 128)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q = torch.randn((2, 3, 8, 128), device=DEV).bfloat16()
    a = lib.spec_verify_attn_q8(q, kl, vl, table, lens, layout=layout, num_blocks=nb, H_kv=H)
    assert torch.equal(a, lib.spec_verify_attn_q8(q, dense_k, dense_v, table, lens))


# ----------------------------------------------------------------- gather ---

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,bs,H,lens,start,rows", [
    (128, 16, 2, (1, 16, 17, 300), (0, 0, 0, 0), 300), (128, 16, 8, (77, 40), (60, 3), 17),
    (128, 16, 1, (50,), (-5,), 70), (128, 16, 3, (0, 33), (0, 32), 1), (64, 8, 2, (30, 9), (7, 0), 11),
    (256, 32, 1, (70,), (31,), 40), (96, 24, 2, (50, 1), (1, 1), 55), (128, 16, 5, (130, 64), (127, 2000000000), 16),
    (16, 1, 3, (9,), (2,), 5), (256, 64, 2, (200,), (3,), 190),
])
def test_gather_is_exact(lib, dtype, d, bs, H, lens, start, rows):
    table, total = table_for(lens, bs, seed=rows)
    kc, vc = q8_pools(total, H, d, bs, seed=rows)
    st = status0()
    got = lib.kv_block_gather_q8(kc.to(DEV), vc.to(DEV), table.to(DEV), i32(lens), i32(start), rows, d, block_size=bs,
                                 out_dtype=dtype, status=st, H_kv=H)
    assert int(st) == 0
    for pool, out in zip((kc, vc), got):
        want = np.zeros((len(lens), rows, H, d))
        for b, L in enumerate(lens):
            v = oq8.dense(pool.numpy(), table[b].numpy(), L, H, d, bs)
            for i in range(rows):
                if 0 <= start[b] + i < L:
                    want[b, i] = v[start[b] + i]
        assert np.array_equal(out.cpu().double().numpy(), want)


def test_gather_of_other_scales(lib):
    # a scale that is no power of two: the rounding to the output type, and in f32 the product's
    kc, vc = q8_pools(2, 2, 128, 16, seed=4, spread=False)
    for pool in (kc, vc):
        lib.q8_views(pool, 2, 128)[1][:] = torch.tensor([0.3, 1e-12])
    for dtype in (torch.bfloat16, torch.float32):
        got = lib.kv_block_gather_q8(kc.to(DEV), vc.to(DEV), i32([[1, 0]]), i32([32]), i32([0]), 32, 128, out_dtype=dtype)
        for pool, out in zip((kc, vc), got):
            want = oq8.dense(pool.numpy(), [1, 0], 32, 2, 128)
            err = np.abs(out.cpu().double().numpy()[0] - want)
            assert (err <= (torch.finfo(dtype).eps / 2 + 2.0 ** -24) * np.abs(want)).all()


def test_gather_bad_lengths_and_blocks_give_zero_rows(lib):
    kc, vc = (p.to(DEV) for p in q8_pools(6, 2, 128, 16, seed=5))
    st = status0()
    table = i32([[0, 99], [1, 2], [3, 4]])
    k, v = lib.kv_block_gather_q8(kc, vc, table, i32([32, 33, -1]), i32([0, 0, 0]), 32, 128, status=st)
    assert int(st) == 1 | 2
    assert (k[0, 16:] == 0).all() and (v[0, 16:] == 0).all() and (k[1:] == 0).all() and (v[1:] == 0).all()
    good, _ = lib.kv_block_gather_q8(kc, vc, table, i32([16, 16, 16]), i32([0, 0, 0]), 16, 128)
    assert torch.equal(k[0, :16], good[0])
    k, v = lib.kv_block_gather_q8(kc, vc, table, i32([16, 16, 16]), i32([0, 0, 0]), 0, 128)
    assert k.shape == (3, 0, 2, 128)


# -------------------------------------------------------------- attention ---

SHAPES = [
    # H_q, H_kv, n_new, lengths
    (32, 8, 1, (1, 16, 1000)), (8, 8, 1, (127, 128, 129, 2)), (64, 8, 5, (5, 300, 517)), (64, 8, 8, (700, 8)),
    (16, 1, 8, (129, 640)), (28, 4, 3, (255, 3, 257, 90)), (16, 2, 9, (1100, 9)), (4, 4, 33, (33, 150)),
    (2, 1, 64, (64, 400)), (12, 2, 4, (64,)),
]
WINDOWS = [(0, 0), (1, 0), (5, 3), (16, 16), (100, 17), (129, 64), (300, 1), (37, 5000), (2 ** 31 - 1, 4)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("H_q,H_kv,n,lens", SHAPES)
def test_attention(lib, H_q, H_kv, n, lens, window, sinks):
    table, total = table_for(lens, 16, seed=n, max_blocks=-(-max(lens) // 16) + 1)
    kc, vc = q8_pools(total, H_kv, 128, 16, seed=n + H_q)
    q = torch.randn((len(lens), n, H_q, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    st = status0()
    out = lib.spec_verify_attn_q8(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32(lens), window=window,
                                  sinks=sinks, status=st)
    assert int(st) == 0
    check_q8_attention(out, *q8_reference(q, kc, vc, table, lens, H_kv, 16, window, sinks))


@pytest.mark.parametrize("window,sinks", [(0, 0), (33, 5), (200, 40)])
@pytest.mark.parametrize("H_q,H_kv,n", [(2, 2, r) for r in (9, 13, 24, 40, 47, 49, 57, 65, 97, 101, 128, 200)] + [(24, 2, 5), (20, 1, 5), (48, 1, 7)])
def test_attention_query_rows(lib, H_q, H_kv, n, window, sinks):
    # every way the query rows of a kv head are dealt to row groups and warpgroups
    lens = [n, n + 1, 300, 129 + n, 1025]
    table, total = table_for(lens, 16, seed=n)
    kc, vc = q8_pools(total, H_kv, 128, 16, seed=n + H_q)
    q = torch.randn((len(lens), n, H_q, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    st = status0()
    out = lib.spec_verify_attn_q8(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32(lens), window=window,
                                  sinks=sinks, status=st)
    assert int(st) == 0
    check_q8_attention(out, *q8_reference(q, kc, vc, table, lens, H_kv, 16, window, sinks))


@pytest.mark.parametrize("window,sinks", [(0, 0), (7, 3), (40, 20)])
@pytest.mark.parametrize("d,bs,H_q,H_kv,n,lens,qd", [
    (64, 16, 8, 2, 5, (70, 5), torch.bfloat16), (96, 8, 4, 4, 2, (33, 2), torch.bfloat16),
    (256, 32, 4, 1, 3, (130, 64), torch.bfloat16), (128, 32, 8, 2, 4, (100,), torch.bfloat16),
    (128, 16, 8, 2, 4, (100, 4, 250), torch.float32), (16, 7, 2, 1, 1, (1, 50), torch.float32),
    (128, 16, 36, 1, 4, (100, 20), torch.bfloat16),
])
def test_attention_other_shapes(lib, d, bs, H_q, H_kv, n, lens, qd, window, sinks):
    table, total = table_for(lens, bs, seed=n)
    kc, vc = q8_pools(total, H_kv, d, bs, seed=n + H_q)
    q = torch.randn((len(lens), n, H_q, d), generator=torch.Generator().manual_seed(9)).to(qd)
    st = status0()
    out = lib.spec_verify_attn_q8(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32(lens), window=window,
                                  sinks=sinks, block_size=bs, status=st, H_kv=H_kv)
    assert int(st) == 0
    check_q8_attention(out, *q8_reference(q, kc, vc, table, lens, H_kv, bs, window, sinks))


@pytest.mark.parametrize("window,sinks", [(0, 0), (1500, 20)])
@pytest.mark.parametrize("B,H_q,H_kv,n,lo,hi", [(40, 64, 8, 5, 5, 3000), (3, 16, 2, 1, 20000, 40000),
                                                (300, 8, 2, 2, 2, 400), (1, 64, 8, 8, 60001, 60001)])
def test_attention_large(lib, B, H_q, H_kv, n, lo, hi, window, sinks):
    lens = torch.randint(lo, hi + 1, (B,), generator=torch.Generator().manual_seed(B)).tolist()
    table, total = table_for(lens, 16, seed=2)
    kc, vc = q8_pools(total, H_kv, 128, 16, seed=3, spread=False)
    q = torch.randn((B, n, H_q, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    st = status0()
    out = lib.spec_verify_attn_q8(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32(lens), window=window,
                                  sinks=sinks, status=st)
    assert int(st) == 0 and torch.isfinite(out).all()
    rows = sorted({0, B // 2, B - 1, int(np.argmax(lens)), int(np.argmin(lens))})[:4]
    check_q8_attention(out, *q8_reference(q, kc, vc, table, lens, H_kv, 16, window, sinks, rows), rows=rows)


@pytest.mark.parametrize("H_q,H_kv,n", [(32, 8, 1), (64, 8, 5), (16, 1, 2), (64, 8, 8)])
def test_attention_many_short_sequences(lib, H_q, H_kv, n):
    # far more sequences than CTAs, most of them a part of one tile, some empty or with a bad length
    B = 500
    lens = torch.randint(n, 200, (B,), generator=torch.Generator().manual_seed(n)).tolist()
    lens[7::50] = [2000] * 10
    table, total = table_for(lens, 16, seed=2)
    bad = {3: 0, 4: -5, 100: n - 1, 499: 16 * table.shape[1] + 1}
    kc, vc = q8_pools(total, H_kv, 128, 16, seed=3, spread=False)
    q = torch.randn((B, n, H_q, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    given = [bad.get(b, L) for b, L in enumerate(lens)]
    st = status0()
    out = torch.full_like(q, 7.0, device=DEV)
    lib.spec_verify_attn_q8(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32(given), out=out, status=st)
    assert int(st) == 1
    assert (out[list(bad)] == 7).all()
    rows = [b for b in range(B) if b not in bad]
    check_q8_attention(out, *q8_reference(q, kc, vc, table, lens, H_kv, 16, rows=rows), rows=rows)


def test_attention_bad_lengths_and_blocks(lib):
    kc, vc = (p.to(DEV) for p in q8_pools(8, 2, 128, 16, seed=5, spread=False))
    q = torch.randn((4, 4, 8, 128), device=DEV).bfloat16()
    table = i32([[0, 1], [2, 99], [4, 5], [6, 7]])
    out = torch.full_like(q, 7.0)
    st = status0()
    lib.spec_verify_attn_q8(q, kc, vc, table, i32([3, 32, 33, 30]), out=out, status=st)
    assert int(st) == 1 | 2
    assert (out[0] == 7).all() and (out[2] == 7).all()   # rows of sequences with a bad length stay as they were
    good = lib.spec_verify_attn_q8(q[3:], kc, vc, table[3:], i32([30]))
    assert torch.allclose(out[3].float(), good[0].float(), atol=2e-2)


@pytest.mark.parametrize("qd", [torch.bfloat16, torch.float32])
def test_attention_window_reads_no_other_pages(lib, qd):
    # table entries of released pages are -1, and what the read blocks hold outside the window and sinks is NaN
    L, n, W, S = 500, 3, 50, 18
    table, total = table_for([L], 16, seed=4)
    kc, vc = q8_pools(total, 2, 128, 16, seed=6, spread=False)
    q = torch.randn((1, n, 8, 128), generator=torch.Generator().manual_seed(9)).to(qd)
    ref, A = q8_reference(q, kc, vc, table, [L], 2, 16, W, S)
    t = np.arange(L)
    hidden = (t >= S) & (t <= L - n - W)
    for blk in range(table.shape[1]):
        here = np.flatnonzero(hidden[blk * 16:(blk + 1) * 16])
        if len(here) == 16:
            table[0, blk] = -1
        else:
            for pool in (kc, vc):
                lib.q8_views(pool, 2, 128)[0].view(torch.uint8)[int(table[0, blk])][:, here] = 0x7F
    st = status0()
    out = lib.spec_verify_attn_q8(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32([L]), window=W, sinks=S, status=st)
    assert int(st) == 0
    check_q8_attention(out, ref, A)


@pytest.mark.parametrize("L", [37, 33, 48, 128, 129, 250, 300])
@pytest.mark.parametrize("H_q,n", [(8, 2), (16, 8), (64, 8)])
def test_attention_garbage_past_the_end(lib, H_q, n, L):
    # unwritten slots of the last page hold NaN codes
    table, total = table_for([L, 200], 16, seed=4)
    kc, vc = q8_pools(total, 2, 128, 16, seed=6, spread=False)
    q = torch.randn((2, n, H_q, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    ref, A = q8_reference(q, kc, vc, table, [L, 200], 2, 16)
    for pool in (kc, vc):
        codes = lib.q8_views(pool, 2, 128)[0].view(torch.uint8)
        if L % 16:
            codes[int(table[0, L // 16]), :, L % 16:] = 0x7F
        codes[int(table[1, 12]), :, 8:] = 0xFF
    out = lib.spec_verify_attn_q8(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32([L, 200]))
    check_q8_attention(out, ref, A)


def test_attention_zeroed_pool(lib):
    # pages that were never written (scale 0): every value is 0
    kc, vc = lib.alloc_q8_pools(4, 2, 128)
    out = lib.spec_verify_attn_q8(torch.randn((1, 2, 8, 128), device=DEV).bfloat16(), kc, vc, i32([[1, 3]]), i32([20]))
    assert (out == 0).all()


def test_attention_scales_of_other_kinds(lib):
    # pages filled elsewhere: any positive scale; zero, negative, NaN read as the smallest, infinity as the largest
    H, L = 2, 400
    table, total = table_for([L], 16, seed=4)
    kc, vc = q8_pools(total, H, 128, 16, seed=6, spread=False)
    rng = np.random.default_rng(1)
    for pool, lo in ((kc, 0.5), (vc, 0.1)):
        s = lib.q8_views(pool, H, 128)[1]
        s *= torch.from_numpy((lo + rng.random(s.shape)).astype(np.float32))
    s = lib.q8_views(vc, H, 128)[1]
    s[int(table[0, 3])], s[int(table[0, 4])], s[int(table[0, 5])] = 0.0, float("nan"), -1.0
    q = torch.randn((1, 3, 16, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    ref, A = q8_reference(q, kc, vc, table, [L], H, 16)
    out = lib.spec_verify_attn_q8(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32([L]))
    check_q8_attention(out, ref, A)


def test_attention_nan_query_stays_in_its_row(lib):
    table, total = table_for([200], 16, seed=4)
    kc, vc = (p.to(DEV) for p in q8_pools(total, 2, 128, 16, seed=6, spread=False))
    q = torch.randn((1, 3, 8, 128), device=DEV).bfloat16()
    good = lib.spec_verify_attn_q8(q, kc, vc, table.to(DEV), i32([200]))
    q[0, 1, 2, 5], q[0, 2, 7, 0] = float("nan"), float("inf")
    out = lib.spec_verify_attn_q8(q, kc, vc, table.to(DEV), i32([200]))
    bad = torch.zeros(1, 3, 8, dtype=torch.bool, device=DEV)
    bad[0, 1, 2] = bad[0, 2, 7] = True
    assert torch.equal(out[~bad], good[~bad]) and torch.isnan(out[0, 1, 2]).all()


def test_far_pages(lib):
    # pages past 2^31 bytes of a pool
    nb = 140_000
    page = lib.q8_page_bytes(8, 128)
    pool_k, pool_v = (torch.empty((nb, page), dtype=torch.uint8, device=DEV) for _ in range(2))
    assert pool_k.numel() > 2 ** 31
    ids = [nb - 1, 0, nb - 2, 135_001]
    kc, vc = q8_pools(4, 8, 128, 16, seed=6)
    pool_k[torch.tensor(ids)], pool_v[torch.tensor(ids)] = kc.to(DEV), vc.to(DEV)
    q = torch.randn((1, 2, 32, 128), device=DEV).bfloat16()
    small = i32([[0, 1, 2, 3]])
    assert torch.equal(lib.spec_verify_attn_q8(q, pool_k, pool_v, i32([ids]), i32([60])),
                       lib.spec_verify_attn_q8(q, kc.to(DEV), vc.to(DEV), small, i32([60])))
    a = lib.kv_block_gather_q8(pool_k, pool_v, i32([ids]), i32([60]), i32([0]), 60, 128)
    b = lib.kv_block_gather_q8(kc.to(DEV), vc.to(DEV), small, i32([60]), i32([0]), 60, 128)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    new = torch.randn((1, 30, 8, 128), device=DEV).bfloat16()
    lib.kv_block_append_q8(new, new, pool_k, pool_v, i32([ids]), i32([60]))
    kd, vd = kc.to(DEV), vc.to(DEV)
    lib.kv_block_append_q8(new, new, kd, vd, small, i32([60]))
    assert torch.equal(pool_k[torch.tensor(ids)], kd) and torch.equal(pool_v[torch.tensor(ids)], vd)


def test_attention_is_deterministic_and_shares_a_workspace(lib):
    lens = [3000, 17, 900, 64]
    table, total = table_for(lens, 16, seed=2)
    kc, vc = (p.to(DEV) for p in q8_pools(total, 8, 128, 16, seed=3, spread=False))
    q = torch.randn((4, 5, 64, 128), device=DEV).bfloat16()
    ws = lib.alloc_workspace(lib.attn_q8_workspace_size(4, 5, 64, 8, 128, table.shape[1]), DEV)
    ws.random_(0, 256)   # contents need no initialisation
    a = lib.spec_verify_attn_q8(q, kc, vc, table.to(DEV), i32(lens), workspace=ws)
    for _ in range(5):
        assert torch.equal(a, lib.spec_verify_attn_q8(q, kc, vc, table.to(DEV), i32(lens), workspace=ws))


# ---------------------------------------------------------------- together ---

def test_graphs_that_share_a_workspace(lib):
    # two rounds (rotation, append, attention) captured as graphs over one workspace, replayed in turn on a side stream,
    # follow changed inputs
    lens = [i32([700, 33]), i32([90, 410])]
    table, total = table_for([720, 420], 16, seed=2)
    table = table.to(DEV)
    start = [p.to(DEV) for p in q8_pools(total, 2, 128, 16, seed=3, spread=False)]
    kc, vc = (p.clone() for p in start)
    new = torch.randn((2, 3, 2, 128), device=DEV).bfloat16()
    q = torch.randn((2, 3, 16, 128), device=DEV).bfloat16()
    qr, nr = torch.empty_like(q), torch.empty_like(new)
    rope = lib.Rope(128)
    ws = lib.alloc_workspace(lib.attn_q8_workspace_size(2, 3, 16, 2, 128, table.shape[1]), DEV)
    outs = [torch.empty_like(q) for _ in lens]

    def one(i):
        lib.spec_rope(q, new, rope, seq_lens=lens[i], q_out=qr, k_out=nr)
        lib.kv_block_append_q8(nr, new, kc, vc, table, lens[i])
        lib.spec_verify_attn_q8(qr, kc, vc, table, lens[i], window=300, sinks=4, out=outs[i], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for i in range(2):
            one(i)
        torch.cuda.synchronize()
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                one(i)
            graphs.append(g)
    q.normal_()
    new.normal_()
    kc.copy_(start[0])
    vc.copy_(start[1])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for g in graphs + graphs:
            g.replay()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    pools = [kc.clone(), vc.clone()]
    kc.copy_(start[0])
    vc.copy_(start[1])
    for i in (0, 1, 0, 1):
        one(i)
        torch.cuda.synchronize()
    assert torch.equal(kc, pools[0]) and torch.equal(vc, pools[1])
    for i in range(2):
        assert torch.equal(outs[i], got[i])
        qi, _ = lib.spec_rope(q, None, rope, seq_lens=lens[i])
        check_q8_attention(got[i], *q8_reference(qi, kc, vc, table, lens[i].tolist(), 2, 16, 300, 4))


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("B,H,rows", [(1, 2, 40), (4, 8, 333), (16, 8, 1024)])
def test_rows_move_between_caches_without_a_wait(lib, captured, B, H, rows):
    # read back, rotated in place, appended elsewhere, nothing between: bit-equal to the same with synchronisations
    lens = [rows] * B
    table, total = table_for(lens, 16, seed=rows)
    table, L = table.to(DEV), i32(lens)
    src = [p.to(DEV) for p in q8_pools(min(total, 40), H, 128, 16, seed=3, spread=False)]
    table = table % src[0].shape[0]   # (read only: sequences may share pages)
    own = table_for(lens, 16, seed=rows + 1)[0].to(DEV)
    start = torch.zeros_like(L)
    buf = [torch.empty((B, rows, H, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    rope = lib.Rope(128)
    q = torch.randn((B, 2, 4 * H, 128), device=DEV).bfloat16()

    def move(dst, wait):
        outs = []
        for window in (0, 100):
            for pair in (src, src[::-1]):
                lib.kv_block_gather_q8(*pair, table, L, start, rows, 128, k_out=buf[0], v_out=buf[1])
                wait()
                lib.spec_rope(None, buf[0], rope, seq_lens=L, k_out=buf[0])
                wait()
                lib.kv_block_append_q8(*buf, *dst, own, L)
                wait()
                outs.append(lib.spec_verify_attn_q8(q, *dst, own, L, window=window))
                wait()
        return outs

    want_pool = lib.alloc_q8_pools(total, H, 128)
    want = move(want_pool, torch.cuda.synchronize)
    pool = lib.alloc_q8_pools(total, H, 128)
    got = move(pool, lambda: None)
    if captured:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = move(pool, lambda: None)
    for _ in range(3):
        for t in (*pool, *buf):
            t.zero_()
        if captured:
            g.replay()
        else:
            got = move(pool, lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(pool[0], want_pool[0]) and torch.equal(pool[1], want_pool[1])


def test_verify_step_and_layers(lib):
    # verify_step and MultiLayerVerify (captured, replayed) over 8-bit, 4-bit and plain layers, with and without a rope
    import workloads
    cfg = workloads.CONFIGS["tiny"].with_(kv_dtype="bf16", q_dtype="bf16", d_head=128, logit_dtype="bf16",
                                          ctx=("fixed", (250, 77)))
    a = {k: (t.to(DEV) if isinstance(t, torch.Tensor) else t) for k, t in
         {**workloads.make_attention_inputs(cfg, 0), **workloads.make_append_inputs(cfg, 0),
          **workloads.make_sampling_inputs(cfg, 0)}.items()}
    lens = a["seq_lens"].tolist()
    total, n = a["k_cache"].shape[0], a["q"].shape[1]
    first = [p.to(DEV) for p in q8_pools(total, cfg.H_kv, 128, 16, seed=8, spread=False)]
    st = status0()
    rope = lib.Rope(128, theta=500000.0)
    pos = np.array([[L - n + j for j in range(n)] for L in lens])
    for W, S, r in ((0, 0, None), (40, 5, rope)):
        kc, vc = (p.clone() for p in first)
        out, toks, nacc = lib.verify_step(a["q"], a["k_new"], a["v_new"], kc, vc, a["block_table"], a["seq_lens"],
                                          a["target_logits"], a["draft_logits"], a["draft_tokens"], a["uniforms"],
                                          status=st, window=W, sinks=S, rope=r)
        q, k = a["q"], a["k_new"]
        if r is not None:   # the rotated rows by the oracle, to a rounding, then the append's bits from the kernel's rows
            want = orope.rotate(q.cpu().double().numpy(), pos, np.array(r.inv_freq))
            q, k = lib.spec_rope(q, k, r, seq_lens=a["seq_lens"])
            assert np.abs(q.cpu().double().numpy() - want).max() <= 2.0 ** -8 * np.abs(want).max()
        ref = oq8.append(first[0].cpu().numpy(), first[1].cpu().numpy(), k.cpu().float().numpy(), a["v_new"].cpu().float().numpy(),
                         a["block_table"].cpu().numpy(), lens)
        assert np.array_equal(kc.cpu().numpy(), ref[0]) and np.array_equal(vc.cpu().numpy(), ref[1])
        check_q8_attention(out, *q8_reference(q, kc, vc, a["block_table"], lens, cfg.H_kv, 16, W, S))
    ref_toks = lib.spec_verify_sample(a["target_logits"], a["draft_logits"], a["draft_tokens"], a["uniforms"])[0]
    assert int(st) == 0 and torch.equal(toks, ref_toks)
    common = dict(q=a["q"], k_new=a["k_new"], v_new=a["v_new"])
    k4, v4 = lib.alloc_q4_pools(total, cfg.H_kv, 128)
    layers = [dict(common, k_cache=first[0].clone(), v_cache=first[1].clone(), rope=rope),
              dict(common, k_cache=first[0].clone(), v_cache=first[1].clone(), window=64, sinks=4),
              dict(common, k_cache=k4, v_cache=v4),
              dict(common, k_cache=a["k_cache"].clone(), v_cache=a["v_cache"].clone(), rope=rope, window=30),
              dict(common, k_cache=a["k_cache"], v_cache=a["v_cache"])]
    m = lib.MultiLayerVerify(layers, a["block_table"], a["seq_lens"], a["target_logits"], a["draft_logits"],
                             a["draft_tokens"], a["uniforms"])
    m.run()
    torch.cuda.synchronize()
    want = [o.clone() for o in m.outs]
    for l, o in zip(layers, want):   # each layer by its own calls
        q, _ = lib.spec_rope(a["q"], None, rope, seq_lens=a["seq_lens"]) if l.get("rope") else (a["q"], None)
        one = lib._attn_any(q, l["k_cache"], l["v_cache"], a["block_table"], a["seq_lens"], None, None, None, l.get("window", 0),
                            l.get("sinks", 0), 16, None, None, None)
        assert torch.equal(one, o)
    m.capture()
    for o in m.outs:
        o.fill_(float("nan"))
    m.replay()
    torch.cuda.synchronize()
    assert int(m.status) == 0 and torch.equal(m.out_tokens, ref_toks)
    for o, w in zip(m.outs, want):
        assert torch.equal(o, w)
    check_q8_attention(m.outs[1], *q8_reference(a["q"], layers[1]["k_cache"], layers[1]["v_cache"], a["block_table"], lens,
                                                cfg.H_kv, 16, 64, 4))


def test_tree_step_with_a_rope(lib):
    # the rotation by depth, then the tree's round: the same as rotating beforehand
    B, n, H_q, H, V, nb = 2, 5, 8, 2, 50, 12
    g = torch.Generator().manual_seed(3)
    parent = i32([[-1, 0, 0, 1, 2], [-1, 0, 1, 2, 2]])
    depth = i32([[0, 1, 1, 2, 2], [0, 1, 2, 3, 3]])
    lens, table = i32([40, 70]), i32([[0, 1, 2, 3, 4], [5, 6, 7, 8, 9]])
    q, k, v = (torch.randn((B, n, h, 128), generator=g).bfloat16().to(DEV) for h in (H_q, H, H))
    pools = [torch.randn((nb, H, 16, 128), generator=g).bfloat16().to(DEV) for _ in range(2)]
    logits = torch.randn((2, B, n, V), generator=g).to(DEV)
    toks = torch.randint(0, V, (B, n), generator=g).to(torch.int32).to(DEV)
    u = torch.rand((B, n, 2), generator=g).to(DEV)
    rope = lib.Rope(128)
    pos = (lens[:, None] - n + depth).contiguous()
    a = [p.clone() for p in pools]
    got = lib.tree_verify_step(q, k, v, *a, table, lens, parent, logits[0].contiguous(), logits[1].contiguous(), toks, u, rope=rope,
                               positions=pos)
    b = [p.clone() for p in pools]
    qr, kr = lib.spec_rope(q, k, rope, positions=pos)
    want = lib.tree_verify_step(qr, kr, v, *b, table, lens, parent, logits[0].contiguous(), logits[1].contiguous(), toks, u)
    for x, y in zip((*got, *a), (*want, *b)):
        assert torch.equal(x, y)


def test_rounds_with_the_block_manager(lib):
    # forks, copy-on-write of 8-bit pages, appends, rollbacks: pages and rows equal a model that keeps every sequence's pages apart
    bm = lib.BlockManager(40)
    H = 2
    kc, vc = lib.alloc_q8_pools(40, H, 128)
    page = lib.q8_page_bytes(H, 128)
    gen = torch.Generator().manual_seed(3)
    model = {}   # sequence: [k pages, v pages] of its own, and its length

    def grow(ids, n, keep):
        pairs = bm.extend(ids, n)
        lib.copy_blocks([kc, vc], pairs, 40)
        table, lens = bm.block_table(ids, 12, device=DEV)
        k, v = (torch.randn((len(ids), n, H, 128), generator=gen).bfloat16() * 2.0 ** int(torch.randint(-4, 5, (1,), generator=gen))
                for _ in range(2))
        lib.kv_block_append_q8(k.to(DEV), v.to(DEV), kc, vc, table, lens)
        for b, i in enumerate(ids):
            L = model[i][2] + n
            model[i][:2] = oq8.append(model[i][0], model[i][1], k[b:b + 1].float().numpy(), v[b:b + 1].float().numpy(),
                                      np.arange(12)[None], [L])
            model[i][2] = L - n + keep[b]
        bm.commit_verify(ids, n, [x - 1 for x in keep])

    for i in (1, 2):
        bm.allocate(i, 0)
        model[i] = [np.zeros((12, page), np.uint8), np.zeros((12, page), np.uint8), 0]
    grow([1, 2], 21, [21, 21])
    bm.fork(1, 3)
    model[3] = list(model[1])
    grow([1, 3], 5, [2, 4])
    bm.share_prefix(2, 4, 20)
    model[4] = [model[2][0].copy(), model[2][1].copy(), 16]
    grow([2, 3, 4], 5, [1, 5, 3])
    ids = [1, 2, 3, 4]
    table, lens = bm.block_table(ids, 12, device=DEV)
    assert lens.tolist() == [model[i][2] for i in ids]
    rows = int(lens.max())
    got = lib.kv_block_gather_q8(kc, vc, table, lens, torch.zeros_like(lens), rows, 128, out_dtype=torch.float32)
    for b, i in enumerate(ids):
        for out, pool in zip(got, model[i][:2]):
            want = oq8.dense(pool, np.arange(12), model[i][2], H, 128)
            assert np.array_equal(out[b, :len(want)].cpu().double().numpy(), want)
    q = torch.randn((4, 1, 8, 128), device=DEV).bfloat16()
    out = lib.spec_verify_attn_q8(q, kc, vc, table, lens)
    check_q8_attention(out, *q8_reference(q, kc, vc, table, lens.tolist(), H, 16))


def test_softmax_scale_and_streams(lib):
    table, total = table_for([333], 16, seed=4)
    kc, vc = (p.to(DEV) for p in q8_pools(total, 2, 128, 16, seed=6, spread=False))
    q = torch.randn((1, 3, 8, 128), device=DEV).bfloat16()
    # scaling q by 4 and the scale by 1/4 is exact
    a = lib.spec_verify_attn_q8(q, kc, vc, table.to(DEV), i32([333]), softmax_scale=0.05)
    s = torch.cuda.Stream()
    q4 = q * 4
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        b = lib.spec_verify_attn_q8(q4, kc, vc, table.to(DEV), i32([333]), softmax_scale=0.0125)
    s.synchronize()
    assert torch.equal(a, b)
    assert math.isfinite(float(a.float().sum()))
