"""The 4-bit paged cache on the GPU against the oracle: append (bit-exact),
read-back, verify attention, and a run of them together."""
import math

import numpy as np
import pytest
import torch

from oracle import q4 as oq4
from q4_utils import check_q4_attention, q4_pools, q4_reference, table_for

pytestmark = pytest.mark.gpu
DEV = "cuda"


def status0():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def same_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))   # (NaN payloads included)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ----------------------------------------------------------------- append ---

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,bs,H,n,lens", [
    (128, 16, 2, 1, (1, 16, 17, 300)), (128, 16, 8, 5, (5, 20, 21, 35)), (128, 16, 1, 37, (37, 50, 64)),
    (128, 16, 3, 200, (200, 333)), (64, 8, 2, 3, (3, 8, 30)), (96, 16, 2, 19, (19, 40)), (256, 32, 1, 70, (70, 101)),
    (32, 64, 2, 64, (64, 65, 100)), (160, 24, 1, 9, (9, 30)),
])
def test_append_is_bit_exact(lib, dtype, d, bs, H, n, lens):
    table, total = table_for(lens, bs, seed=d + n, max_blocks=-(-max(lens) // bs) + 2)
    kc, vc = q4_pools(total, H, d, bs, seed=n)
    g = torch.Generator().manual_seed(7)
    k, v = (torch.randn((len(lens), n, H, d), generator=g).to(dtype) * f for f in (1.0, 3.0))
    k[0, 0, 0], v[0, 0, 0, :7] = 0.25, 100.0
    kd, vd = kc.to(DEV), vc.to(DEV)
    st = status0()
    lib.kv_block_append_q4(k.to(DEV), v.to(DEV), kd, vd, table.to(DEV), i32(lens), block_size=bs, status=st)
    want = oq4.append(kc.numpy(), vc.numpy(), k.float().numpy(), v.float().numpy(), table.numpy(), lens, bs)
    assert int(st) == 0
    for got, ref in zip((kd, vd), want):
        assert np.array_equal(got.cpu().numpy(), ref)


def test_append_special_values(lib):
    # NaN, infinities, constant, zero and huge rows: codes and pairs stay finite and follow the definition
    x = torch.randn((1, 8, 1, 128), generator=torch.Generator().manual_seed(1))
    x[0, 0] = 0.0
    x[0, 1] = float("nan")
    x[0, 2, 0, 5], x[0, 2, 0, 9] = float("nan"), float("inf")
    x[0, 3, 0, 0] = -float("inf")
    x[0, 4] = 3e38
    x[0, 5] *= 1e-30
    x[0, 6] = -7.0
    x[0, 7] *= 1e6
    table, lens = torch.tensor([[2]], dtype=torch.int32), [8]
    kc, vc = q4_pools(3, 1, 128, 16, seed=3)
    kd, vd = kc.to(DEV), vc.to(DEV)
    lib.kv_block_append_q4(x.to(DEV), -x.to(DEV), kd, vd, table.to(DEV), i32(lens))
    want = oq4.append(kc.numpy(), vc.numpy(), x.numpy(), -x.numpy(), table.numpy(), lens)
    assert np.array_equal(kd.cpu().numpy(), want[0]) and np.array_equal(vd.cpu().numpy(), want[1])
    back, _ = lib.kv_block_gather_q4(kd, vd, table.to(DEV), i32(lens), i32([0]), 8, 128, out_dtype=torch.float32)
    assert torch.isfinite(back).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_ties(lib, dtype):
    # values on and next to the middle between two codes, for scales of every kind of mantissa
    g = torch.Generator().manual_seed(2)
    s = torch.rand((64, 1), generator=g) * 3 + 0.01
    half = torch.arange(128) % 31 / 2.0
    x = half[None, :] * s
    x[:32] = half[None, :] * torch.tensor([1.0, 0.5, 3.0, 7.0]).repeat(8)[:, None]
    x[32:48] = torch.nextafter(x[32:48], torch.full((), 100.0))
    x += torch.tensor([0.0, 1.0, -2.5, 0.125]).repeat(16)[:, None]
    x[:, 0], x[:, 30] = x.min(-1).values, x.max(-1).values
    x = x[None, :, None].contiguous().to(dtype)
    table, lens = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32), [64]
    kc, vc = q4_pools(4, 1, 128, 16, seed=3)
    kd, vd = kc.to(DEV), vc.to(DEV)
    lib.kv_block_append_q4(x.to(DEV), (-x).to(DEV), kd, vd, table.to(DEV), i32(lens))
    want = oq4.append(kc.numpy(), vc.numpy(), x.float().numpy(), -x.float().numpy(), table.numpy(), lens)
    assert np.array_equal(kd.cpu().numpy(), want[0]) and np.array_equal(vd.cpu().numpy(), want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_at_any_element(lib, dtype):
    # new rows and read-back buffers that start at an odd element of their storage
    H, n, lens = 3, 21, [40, 21]
    table, total = table_for(lens, 16, seed=5)
    kc, vc = (p.to(DEV) for p in q4_pools(total, H, 128, 16, seed=5))
    k2, v2 = kc.clone(), vc.clone()
    size = 2 * n * H * 128
    flat = torch.randn(2 * size + 8, generator=torch.Generator().manual_seed(5)).to(dtype).to(DEV)
    k, v = (flat[o:o + size].view(2, n, H, 128) for o in (1, size + 3))
    lib.kv_block_append_q4(k, v, kc, vc, table.to(DEV), i32(lens))
    lib.kv_block_append_q4(k.clone(), v.clone(), k2, v2, table.to(DEV), i32(lens))
    assert torch.equal(kc, k2) and torch.equal(vc, v2)
    dst = torch.full((2 * size + 8,), 7.0, dtype=dtype, device=DEV)
    out = [dst[o:o + size].view(2, n, H, 128) for o in (1, size + 3)]
    start = i32([25, -4])
    lib.kv_block_gather_q4(kc, vc, table.to(DEV), i32(lens), start, n, 128, k_out=out[0], v_out=out[1])
    want = lib.kv_block_gather_q4(kc, vc, table.to(DEV), i32(lens), start, n, 128, out_dtype=dtype)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert (dst[[0, size + 1, size + 2] + list(range(2 * size + 3, 2 * size + 8))] == 7).all()


def test_append_bad_lengths_and_blocks_leave_the_pools(lib):
    table = torch.tensor([[0, 1], [99, 99], [2, 3], [4, -1]], dtype=torch.int32, device=DEV)
    kc, vc = (p.to(DEV) for p in q4_pools(6, 2, 128, 16, seed=5))
    k0, v0 = kc.clone(), vc.clone()
    new = torch.randn((4, 4, 2, 128), device=DEV)
    st = status0()
    # shorter than n_new; a block outside the pool; longer than the table; a block of -1
    lib.kv_block_append_q4(new, new, kc, vc, table, i32([3, 20, 33, 20]), status=st)
    assert int(st) == 1 | 2
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_append_strided_records(lib):
    # records of one layer inside a pool of [num_blocks][layers][H_kv][record]
    rec, H, nb, layers = 1088, 2, 7, 3
    big_k, big_v = (torch.randint(0, 256, (nb, layers, H, rec), dtype=torch.uint8, device=DEV) for _ in range(2))
    k0, v0 = big_k.clone(), big_v.clone()
    new = torch.randn((2, 20, H, 128), device=DEV).bfloat16()
    table, lens = i32([[1, 4, 6], [5, 0, 2]]), i32([25, 40])
    layout = (layers * H * rec, rec, 0)
    kl, vl = big_k.view(-1)[H * rec:], big_v.view(-1)[H * rec:]
    lib.kv_block_append_q4(new, new, kl, vl, table, lens, layout=layout, num_blocks=nb)
    dense_k, dense_v = k0[:, 1].contiguous(), v0[:, 1].contiguous()
    lib.kv_block_append_q4(new, new, dense_k, dense_v, table, lens)
    k0[:, 1], v0[:, 1] = dense_k, dense_v
    assert torch.equal(big_k, k0) and torch.equal(big_v, v0)
    start = i32([3, 17])
    a = lib.kv_block_gather_q4(kl, vl, table, lens, start, 9, 128, layout=layout, num_blocks=nb, H_kv=H)
    b = lib.kv_block_gather_q4(dense_k, dense_v, table, lens, start, 9, 128)
    assert same_bits(a[0], b[0]) and same_bits(a[1], b[1])
    q = torch.randn((2, 3, 8, 128), device=DEV).bfloat16()
    a = lib.spec_verify_attn_q4(q, kl, vl, table, lens, layout=layout, num_blocks=nb, H_kv=H)
    assert same_bits(a, lib.spec_verify_attn_q4(q, dense_k, dense_v, table, lens))


# ----------------------------------------------------------------- gather ---

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,bs,H,lens,start,rows", [
    (128, 16, 2, (1, 16, 17, 300), (0, 0, 0, 0), 300), (128, 16, 8, (77, 40), (60, 3), 17),
    (128, 16, 1, (50,), (-5,), 70), (128, 16, 3, (0, 33), (0, 32), 1), (64, 8, 2, (30, 9), (7, 0), 11),
    (256, 32, 1, (70,), (31,), 40), (96, 24, 2, (50, 1), (1, 1), 55), (128, 16, 5, (130, 64), (127, 2000000000), 16),
])
def test_gather(lib, dtype, d, bs, H, lens, start, rows):
    table, total = table_for(lens, bs, seed=rows)
    kc, vc = q4_pools(total, H, d, bs, seed=rows)
    st = status0()
    got = lib.kv_block_gather_q4(kc.to(DEV), vc.to(DEV), table.to(DEV), i32(lens), i32(start), rows, d, block_size=bs,
                                 out_dtype=dtype, status=st)
    assert int(st) == 0
    for kind, pool, g in zip("kv", (kc, vc), got):
        want = np.zeros((len(lens), rows, H, d))
        size = np.zeros_like(want)
        for b, L in enumerate(lens):
            v = oq4.dense(kind, pool.numpy(), table[b].numpy(), L, d, bs)
            for i in range(rows):
                if 0 <= start[b] + i < L:
                    want[b, i] = v[start[b] + i]
                    size[b, i] = np.abs(v[start[b] + i]) + 2 * np.abs(v[start[b] + i]).max(-1, keepdims=True)
        err = np.abs(g.cpu().double().numpy() - want)
        bound = 2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0
        assert (err <= bound + 2.0 ** -23 * size).all(), err.max()


def test_gather_bad_lengths_and_blocks_give_zero_rows(lib):
    kc, vc = (p.to(DEV) for p in q4_pools(6, 2, 128, 16, seed=5))
    st = status0()
    table = i32([[0, 99], [1, 2], [3, 4]])
    k, v = lib.kv_block_gather_q4(kc, vc, table, i32([32, 33, -1]), i32([0, 0, 0]), 32, 128, status=st)
    assert int(st) == 1 | 2
    assert (k[0, 16:] == 0).all() and (v[0, 16:] == 0).all() and (k[1:] == 0).all() and (v[1:] == 0).all()
    good, _ = lib.kv_block_gather_q4(kc, vc, table, i32([16, 16, 16]), i32([0, 0, 0]), 16, 128)
    assert torch.equal(k[0, :16], good[0])
    k, v = lib.kv_block_gather_q4(kc, vc, table, i32([16, 16, 16]), i32([0, 0, 0]), 0, 128)
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
    kc, vc = q4_pools(total, H_kv, 128, 16, seed=n + H_q)
    q = torch.randn((len(lens), n, H_q, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    st = status0()
    out = lib.spec_verify_attn_q4(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32(lens), window=window,
                                  sinks=sinks, status=st)
    assert int(st) == 0
    check_q4_attention(out, *q4_reference(q, kc, vc, table, lens, 16, window, sinks))


@pytest.mark.parametrize("window,sinks", [(0, 0), (33, 5), (200, 40)])
@pytest.mark.parametrize("H_q,H_kv,n", [(2, 2, r) for r in (47, 49, 57, 65, 97, 101, 128)] + [(24, 2, 5), (20, 1, 5)])
def test_attention_query_rows(lib, H_q, H_kv, n, window, sinks):
    # every way the query rows of a kv head are dealt to row groups and warpgroups
    lens = [n, n + 1, 300, 129 + n, 1025]
    table, total = table_for(lens, 16, seed=n)
    kc, vc = q4_pools(total, H_kv, 128, 16, seed=n + H_q)
    q = torch.randn((len(lens), n, H_q, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    st = status0()
    out = lib.spec_verify_attn_q4(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32(lens), window=window,
                                  sinks=sinks, status=st)
    assert int(st) == 0
    check_q4_attention(out, *q4_reference(q, kc, vc, table, lens, 16, window, sinks))


@pytest.mark.parametrize("window,sinks", [(0, 0), (7, 3), (40, 20)])
@pytest.mark.parametrize("d,bs,H_q,H_kv,n,lens,qd", [
    (64, 16, 8, 2, 5, (70, 5), torch.bfloat16), (96, 8, 4, 4, 2, (33, 2), torch.bfloat16),
    (256, 32, 4, 1, 3, (130, 64), torch.bfloat16), (128, 32, 8, 2, 4, (100,), torch.bfloat16),
    (128, 16, 8, 2, 4, (100, 4, 250), torch.float32), (32, 8, 2, 1, 1, (1, 50), torch.float32),
    (128, 16, 36, 1, 4, (100, 20), torch.bfloat16),
])
def test_attention_other_shapes(lib, d, bs, H_q, H_kv, n, lens, qd, window, sinks):
    table, total = table_for(lens, bs, seed=n)
    kc, vc = q4_pools(total, H_kv, d, bs, seed=n + H_q)
    q = torch.randn((len(lens), n, H_q, d), generator=torch.Generator().manual_seed(9)).to(qd)
    st = status0()
    out = lib.spec_verify_attn_q4(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32(lens), window=window,
                                  sinks=sinks, block_size=bs, status=st)
    assert int(st) == 0
    check_q4_attention(out, *q4_reference(q, kc, vc, table, lens, bs, window, sinks))


@pytest.mark.parametrize("window,sinks", [(0, 0), (1500, 20)])
@pytest.mark.parametrize("B,H_q,H_kv,n,lo,hi", [(40, 64, 8, 5, 5, 3000), (3, 16, 2, 1, 20000, 40000),
                                                (300, 8, 2, 2, 2, 400), (1, 64, 8, 8, 60001, 60001)])
def test_attention_large(lib, B, H_q, H_kv, n, lo, hi, window, sinks):
    lens = torch.randint(lo, hi + 1, (B,), generator=torch.Generator().manual_seed(B)).tolist()
    table, total = table_for(lens, 16, seed=2)
    kc, vc = q4_pools(total, H_kv, 128, 16, seed=3, spread=False)
    q = torch.randn((B, n, H_q, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    st = status0()
    out = lib.spec_verify_attn_q4(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32(lens), window=window,
                                  sinks=sinks, status=st)
    assert int(st) == 0 and torch.isfinite(out).all()
    rows = sorted({0, B // 2, B - 1, int(np.argmax(lens)), int(np.argmin(lens))})[:4]
    check_q4_attention(out, *q4_reference(q, kc, vc, table, lens, 16, window, sinks, rows), rows=rows)


@pytest.mark.parametrize("H_q,H_kv,n", [(32, 8, 1), (64, 8, 5), (16, 1, 2), (64, 8, 8)])
def test_attention_many_short_sequences(lib, H_q, H_kv, n):
    # far more sequences than CTAs, most of them a part of one tile, some empty or with a bad length
    B = 500
    lens = torch.randint(n, 200, (B,), generator=torch.Generator().manual_seed(n)).tolist()
    lens[7::50] = [2000] * 10
    table, total = table_for(lens, 16, seed=2)
    bad = {3: 0, 4: -5, 100: n - 1, 499: 16 * table.shape[1] + 1}
    kc, vc = q4_pools(total, H_kv, 128, 16, seed=3)
    q = torch.randn((B, n, H_q, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    given = [bad.get(b, L) for b, L in enumerate(lens)]
    st = status0()
    out = torch.full_like(q, 7.0, device=DEV)
    lib.spec_verify_attn_q4(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32(given), out=out, status=st)
    assert int(st) == 1
    assert (out[list(bad)] == 7).all()
    rows = [b for b in range(B) if b not in bad]
    check_q4_attention(out, *q4_reference(q, kc, vc, table, lens, 16, rows=rows), rows=rows)


def test_attention_wait_runs_out_then_next_call_is_correct(lib):
    # the code copies are withheld, so every wait on them can only end by its limit (2 ms)
    lens = [700, 5, 3000]
    table, total = table_for(lens, 16, seed=2)
    kc, vc = q4_pools(total, 2, 128, 16, seed=3)
    q = torch.randn((3, 4, 16, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    args = (q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32(lens))
    st = status0()
    try:
        lib.test_hooks(2_000_000, lib.SV_TEST_WITHHOLD_COPIES)
        lib.spec_verify_attn_q4(*args, status=st)
        torch.cuda.synchronize()
    finally:
        lib.test_hooks(0, 0)
    assert int(st) & lib.SV_DEV_TIMEOUT
    st.zero_()
    out = lib.spec_verify_attn_q4(*args, status=st)
    assert int(st) == 0
    check_q4_attention(out, *q4_reference(q, kc, vc, table, lens, 16))


def test_attention_rising_scores_and_extreme_rows(lib):
    # the largest scores come last and grow from tile to tile (every tile moves the running reference), and the
    # queries' rows differ by 2^20 in size
    L, H = 900, 2
    K = torch.randn((1, L, H, 128), generator=torch.Generator().manual_seed(1))
    K += torch.linspace(0, 6, L)[None, :, None, None] * torch.sign(K[:, :1])
    V = torch.randn((1, L, H, 128), generator=torch.Generator().manual_seed(2)) * 100
    V[:, ::7] *= 1e-4
    q = torch.sign(K[:, :1]).repeat_interleave(4, 2).expand(1, 4, 8, 128) * torch.tensor([1.0, 2.0 ** -20, 0.25, 0.0])[None, :, None, None]
    q = q.contiguous().bfloat16()
    table, total = table_for([L], 16, seed=2)
    kc, vc = lib.alloc_q4_pools(total, H, 128)
    lib.kv_block_append_q4(K.to(DEV), V.to(DEV), kc, vc, table.to(DEV), i32([L]))
    out = lib.spec_verify_attn_q4(q.to(DEV), kc, vc, table.to(DEV), i32([L]))
    ref, A = q4_reference(q, kc, vc, table, [L], 16)
    got = out.double().cpu().numpy()
    # scores reach 2^10 here, so the fp32 accumulation's share of the bound is 2^-8 A
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * A).all()


def test_attention_bad_lengths_and_blocks(lib):
    kc, vc = (p.to(DEV) for p in q4_pools(8, 2, 128, 16, seed=5))
    q = torch.randn((4, 4, 8, 128), device=DEV).bfloat16()
    table = i32([[0, 1], [2, 99], [4, 5], [6, 7]])
    out = torch.full_like(q, 7.0)
    st = status0()
    lib.spec_verify_attn_q4(q, kc, vc, table, i32([3, 32, 33, 30]), out=out, status=st)
    assert int(st) == 1 | 2
    assert (out[0] == 7).all() and (out[2] == 7).all()   # rows of sequences with a bad length stay as they were
    good = lib.spec_verify_attn_q4(q[3:], kc, vc, table[3:], i32([30]))
    assert torch.allclose(out[3].float(), good[0].float(), atol=2e-2)


def test_attention_window_reads_no_other_pages(lib):
    # table entries of released pages are -1, and what the read blocks hold outside the window and sinks is NaN
    L, n, W, S = 500, 3, 50, 18
    table, total = table_for([L], 16, seed=4)
    kc, vc = q4_pools(total, 2, 128, 16, seed=6)
    q = torch.randn((1, n, 8, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    ref, A = q4_reference(q, kc, vc, table, [L], 16, W, S)
    t = np.arange(L)
    hidden = (t >= S) & (t <= L - n - W)
    for blk in range(table.shape[1]):
        here = hidden[blk * 16:(blk + 1) * 16]
        if here.all():
            table[0, blk] = -1
        else:
            for pool in (kc, vc):   # NaN pairs
                pairs = pool[int(table[0, blk]), :, 1024:].view(torch.float16).view(-1, 16, 2)
                pairs[:, np.flatnonzero(here)] = float("nan")
    st = status0()
    out = lib.spec_verify_attn_q4(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32([L]), window=W, sinks=S, status=st)
    assert int(st) == 0
    check_q4_attention(out, ref, A)


def test_attention_garbage_past_the_end(lib):
    # unwritten slots of the last page hold NaN pairs
    L = 37
    table, total = table_for([L], 16, seed=4)
    kc, vc = q4_pools(total, 2, 128, 16, seed=6)
    q = torch.randn((1, 2, 8, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    ref, A = q4_reference(q, kc, vc, table, [L], 16)
    for pool in (kc, vc):
        pool[int(table[0, 2]), :, 1024:].view(torch.float16).view(-1, 16, 2)[:, L % 16:] = float("nan")
    out = lib.spec_verify_attn_q4(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32([L]))
    check_q4_attention(out, ref, A)


def test_attention_zeroed_pool(lib):
    # pages that were never written (scale 0): every value is 0
    kc, vc = lib.alloc_q4_pools(4, 2, 128)
    out = lib.spec_verify_attn_q4(torch.randn((1, 2, 8, 128), device=DEV).bfloat16(), kc, vc, i32([[1, 3]]), i32([20]))
    assert (out == 0).all()


def test_attention_nan_query_stays_in_its_row(lib):
    table, total = table_for([200], 16, seed=4)
    kc, vc = (p.to(DEV) for p in q4_pools(total, 2, 128, 16, seed=6, spread=False))
    q = torch.randn((1, 3, 8, 128), device=DEV).bfloat16()
    good = lib.spec_verify_attn_q4(q, kc, vc, table.to(DEV), i32([200]))
    q[0, 1, 2, 5], q[0, 2, 7, 0] = float("nan"), float("inf")
    out = lib.spec_verify_attn_q4(q, kc, vc, table.to(DEV), i32([200]))
    bad = torch.zeros(1, 3, 8, dtype=torch.bool, device=DEV)
    bad[0, 1, 2] = bad[0, 2, 7] = True
    assert torch.equal(out[~bad], good[~bad]) and torch.isnan(out[0, 1, 2]).all()


def test_attention_far_pages(lib):
    # records past 2^31 bytes of a pool
    nb = 260_000
    pool_k, pool_v = (torch.empty((nb, 8, 1088), dtype=torch.uint8, device=DEV) for _ in range(2))
    assert pool_k.numel() > 2 ** 31
    ids = [nb - 1, 0, nb - 2, 250_001]
    kc, vc = q4_pools(4, 8, 128, 16, seed=6)
    pool_k[torch.tensor(ids)], pool_v[torch.tensor(ids)] = kc.to(DEV), vc.to(DEV)
    q = torch.randn((1, 2, 32, 128), device=DEV).bfloat16()
    small = i32([[0, 1, 2, 3]])
    assert torch.equal(lib.spec_verify_attn_q4(q, pool_k, pool_v, i32([ids]), i32([60])),
                       lib.spec_verify_attn_q4(q, kc.to(DEV), vc.to(DEV), small, i32([60])))
    a = lib.kv_block_gather_q4(pool_k, pool_v, i32([ids]), i32([60]), i32([0]), 60, 128)
    b = lib.kv_block_gather_q4(kc.to(DEV), vc.to(DEV), small, i32([60]), i32([0]), 60, 128)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    new = torch.randn((1, 30, 8, 128), device=DEV).bfloat16()
    lib.kv_block_append_q4(new, new, pool_k, pool_v, i32([ids]), i32([60]))
    kd, vd = kc.to(DEV), vc.to(DEV)
    lib.kv_block_append_q4(new, new, kd, vd, small, i32([60]))
    assert torch.equal(pool_k[torch.tensor(ids)], kd) and torch.equal(pool_v[torch.tensor(ids)], vd)


def test_attention_is_deterministic_and_shares_a_workspace(lib):
    lens = [3000, 17, 900, 64]
    table, total = table_for(lens, 16, seed=2)
    kc, vc = (p.to(DEV) for p in q4_pools(total, 8, 128, 16, seed=3, spread=False))
    q = torch.randn((4, 5, 64, 128), device=DEV).bfloat16()
    ws = lib.alloc_workspace(lib.attn_q4_workspace_size(4, 5, 64, 8, 128, table.shape[1]), DEV)
    ws.random_(0, 256)   # contents need no initialisation
    a = lib.spec_verify_attn_q4(q, kc, vc, table.to(DEV), i32(lens), workspace=ws)
    for _ in range(5):
        assert torch.equal(a, lib.spec_verify_attn_q4(q, kc, vc, table.to(DEV), i32(lens), workspace=ws))


# ---------------------------------------------------------------- together ---

def test_graphs_that_share_a_workspace(lib):
    # two rounds captured as graphs over one workspace, replayed in turn on a side stream, follow changed inputs
    lens = [i32([700, 33]), i32([90, 410])]
    table, total = table_for([720, 420], 16, seed=2)
    table = table.to(DEV)
    kc, vc = (p.to(DEV) for p in q4_pools(total, 2, 128, 16, seed=3, spread=False))
    new = torch.randn((2, 3, 2, 128), device=DEV).bfloat16()
    q = torch.randn((2, 3, 16, 128), device=DEV).bfloat16()
    ws = lib.alloc_workspace(lib.attn_q4_workspace_size(2, 3, 16, 2, 128, table.shape[1]), DEV)
    outs = [torch.empty_like(q) for _ in lens]

    def one(i):
        lib.kv_block_append_q4(new, new, kc, vc, table, lens[i])
        lib.spec_verify_attn_q4(q, kc, vc, table, lens[i], window=300, sinks=4, out=outs[i], workspace=ws)

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
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for g in graphs + graphs:
            g.replay()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    for i in range(2):
        one(i)
        torch.cuda.synchronize()
        assert torch.equal(outs[i], got[i])
        ref = q4_reference(q, kc, vc, table, lens[i].tolist(), 16, 300, 4)
        check_q4_attention(got[i], *ref)


def test_verify_step_and_layers_over_4_bit_pools(lib):
    # verify_step and MultiLayerVerify (captured, replayed) over 4-bit, windowed and plain layers
    import workloads
    cfg = workloads.CONFIGS["tiny"].with_(kv_dtype="bf16", q_dtype="bf16", d_head=128, logit_dtype="bf16",
                                          ctx=("fixed", (250, 77)))
    a = {k: (t.to(DEV) if isinstance(t, torch.Tensor) else t) for k, t in
         {**workloads.make_attention_inputs(cfg, 0), **workloads.make_append_inputs(cfg, 0),
          **workloads.make_sampling_inputs(cfg, 0)}.items()}
    lens = a["seq_lens"].tolist()
    total = a["k_cache"].shape[0]
    kc, vc = (p.to(DEV) for p in q4_pools(total, cfg.H_kv, 128, 16, seed=8, spread=False))
    st = status0()
    for W, S in ((0, 0), (40, 5)):
        out, toks, nacc = lib.verify_step(a["q"], a["k_new"], a["v_new"], kc, vc, a["block_table"], a["seq_lens"],
                                          a["target_logits"], a["draft_logits"], a["draft_tokens"], a["uniforms"],
                                          status=st, window=W, sinks=S)
        check_q4_attention(out, *q4_reference(a["q"], kc, vc, a["block_table"], lens, 16, W, S))
    ref_toks = lib.spec_verify_sample(a["target_logits"], a["draft_logits"], a["draft_tokens"], a["uniforms"])[0]
    assert int(st) == 0 and torch.equal(toks, ref_toks)
    common = dict(q=a["q"], k_new=a["k_new"], v_new=a["v_new"])
    layers = [dict(common, k_cache=kc, v_cache=vc), dict(common, k_cache=kc.clone(), v_cache=vc.clone(), window=64, sinks=4),
              dict(common, k_cache=a["k_cache"].clone(), v_cache=a["v_cache"].clone(), window=30),
              dict(common, k_cache=a["k_cache"], v_cache=a["v_cache"])]
    m = lib.MultiLayerVerify(layers, a["block_table"], a["seq_lens"], a["target_logits"], a["draft_logits"],
                             a["draft_tokens"], a["uniforms"])
    m.run()
    torch.cuda.synchronize()
    want = [o.clone() for o in m.outs]
    m.capture()
    for o in m.outs:
        o.fill_(float("nan"))
    m.replay()
    torch.cuda.synchronize()
    assert int(m.status) == 0 and torch.equal(m.out_tokens, ref_toks)
    for o, w in zip(m.outs, want):
        assert torch.equal(o, w)
    check_q4_attention(m.outs[1], *q4_reference(a["q"], layers[1]["k_cache"], layers[1]["v_cache"], a["block_table"], lens,
                                                16, 64, 4))


def test_rounds_with_the_block_manager(lib):
    # forks, copy-on-write of 4-bit pages, appends, rollbacks: every sequence's rows equal a dense model's
    bm = lib.BlockManager(40)
    kc, vc = lib.alloc_q4_pools(40, 2, 128)
    gen = torch.Generator().manual_seed(3)
    model = {}

    def grow(ids, n, keep):
        pairs = bm.extend(ids, n)
        lib.copy_blocks([kc, vc], pairs, 40)
        table, lens = bm.block_table(ids, 12, device=DEV)
        k, v = (torch.randn((len(ids), n, 2, 128), generator=gen).bfloat16() for _ in range(2))
        lib.kv_block_append_q4(k.to(DEV), v.to(DEV), kc, vc, table, lens)
        for b, i in enumerate(ids):
            rows = [oq4.values(*oq4.quantize(x[b].float().numpy()))[:keep[b]] for x in (k, v)]
            model[i] = [np.concatenate((old, r)) for old, r in zip(model[i], rows)]
        bm.commit_verify(ids, n, [x - 1 for x in keep])

    for i in (1, 2):
        bm.allocate(i, 0)
        model[i] = [np.zeros((0, 2, 128))] * 2
    grow([1, 2], 21, [21, 21])
    bm.fork(1, 3)
    model[3] = list(model[1])
    grow([1, 3], 5, [2, 4])
    bm.share_prefix(2, 4, 20)
    model[4] = [x[:16] for x in model[2]]
    grow([2, 3, 4], 5, [1, 5, 3])
    ids = [1, 2, 3, 4]
    table, lens = bm.block_table(ids, 12, device=DEV)
    rows = int(lens.max())
    got = lib.kv_block_gather_q4(kc, vc, table, lens, torch.zeros_like(lens), rows, 128, out_dtype=torch.float32)
    for b, i in enumerate(ids):
        for g, want in zip(got, model[i]):
            assert len(want) == int(lens[b])
            assert np.allclose(g[b, :len(want)].cpu().numpy(), want, rtol=0, atol=1e-6 * np.abs(want).max())
    q = torch.randn((4, 1, 8, 128), device=DEV).bfloat16()
    out = lib.spec_verify_attn_q4(q, kc, vc, table, lens)
    check_q4_attention(out, *q4_reference(q, kc, vc, table, lens.tolist(), 16))


def test_softmax_scale_and_streams(lib):
    table, total = table_for([333], 16, seed=4)
    kc, vc = (p.to(DEV) for p in q4_pools(total, 2, 128, 16, seed=6, spread=False))
    q = torch.randn((1, 3, 8, 128), device=DEV).bfloat16()
    # scaling q by 4 and the scale by 1/4 is exact
    a = lib.spec_verify_attn_q4(q, kc, vc, table.to(DEV), i32([333]), softmax_scale=0.05)
    s = torch.cuda.Stream()
    q4 = q * 4
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        b = lib.spec_verify_attn_q4(q4, kc, vc, table.to(DEV), i32([333]), softmax_scale=0.0125)
    s.synchronize()
    assert torch.equal(a, b)
    assert math.isfinite(float(a.float().sum()))
