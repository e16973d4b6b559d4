"""Verify attention over 4-bit pools where weights and queries span a wide
range: one key that holds most of a long row's weight, and query rows of very
different sizes side by side."""
import math

import pytest
import torch

from q4_utils import check_q4_attention, q4_pools, q4_reference, table_for

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("window,sinks", [(0, 0), (100_000, 4)])
@pytest.mark.parametrize("first", [0, 3])
@pytest.mark.parametrize("L", [9000, 131_000])
def test_one_key_holds_most_of_the_weight(lib, L, first, window, sinks):
    # Eight kv heads; in each, key `first` (of either parity) outweighs every other key 2^gap times, and the others have
    # equal scores (heads 4-7) or scores of one nat's spread. As many sequences as ranges share the pages, so that one
    # range walks a whole row and nothing splits the sums.
    H, B, n, gaps = 8, 19, 2, (14, 17, 20, 23)
    g = torch.Generator().manual_seed(3)
    K = torch.randn((1, L, H, 128), generator=g)
    K[:, :, 4:] = 0.0
    for h in range(H):
        K[:, first, h] = gaps[h % 4] * math.log(2) / math.sqrt(128)   # a constant row: its score is 128 times this
    V = torch.randn((1, L, H, 128), generator=g)
    nb = -(-L // 16)
    table = torch.arange(nb, dtype=torch.int32)[None].to(DEV)
    kc, vc = lib.alloc_q4_pools(nb, H, 128)
    lib.kv_block_append_q4(K.to(DEV), V.to(DEV), kc, vc, table, i32([L]))
    q = torch.ones((B, n, H, 128)).bfloat16()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = lib.spec_verify_attn_q4(q.to(DEV), kc, vc, table.expand(B, -1).contiguous(), i32([L] * B), window=window,
                                  sinks=sinks, status=st)
    assert int(st) == 0
    rows = [0, B - 1]
    ref, A = q4_reference(q, kc, vc, table.expand(B, -1), [L] * B, 16, window, sinks, rows=rows)
    for h in range(H):   # (a head at a time: the norm of one must not hide another's)
        check_q4_attention(out[:, :, h:h + 1], ref[:, :, h:h + 1], A, rows=rows)


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5)])
@pytest.mark.parametrize("H_q,H_kv,n,lens", [(8, 8, 2, (700, 33)), (16, 2, 3, (129, 2000, 3)), (64, 8, 5, (640, 5, 1111)),
                                             (64, 8, 8, (900,)), (32, 1, 4, (500, 77)), (12, 1, 3, (260,))])
@pytest.mark.parametrize("size", [40.0, 70.0, 1e4, 2.0 ** 17, 1e30, 3e38])
def test_query_rows_of_other_sizes_leave_a_row_alone(lib, H_q, H_kv, n, lens, size, window, sinks):
    # the last position's rows (padding of a shorter draft: anything finite) and one head of the first are `size` times larger
    table, total = table_for(lens, 16, seed=n)
    kc, vc = q4_pools(total, H_kv, 128, 16, seed=n + H_q, spread=False)
    q = torch.randn((len(lens), n, H_q, 128), generator=torch.Generator().manual_seed(9)).bfloat16()
    plain = q.clone()
    q[:, -1] = (q[:, -1].float().clamp(-1, 1) * size).bfloat16()
    q[:, 0, 1] = (q[:, 0, 1].float().clamp(-1, 1) * size).bfloat16()
    assert torch.isfinite(q).all()
    good = torch.ones(n, H_q, dtype=torch.bool)
    good[-1] = good[0, 1] = False
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = lib.spec_verify_attn_q4(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32(lens), window=window, sinks=sinks,
                                  status=st)
    assert int(st) == 0
    ref, A = q4_reference(plain, kc, vc, table, lens, 16, window, sinks)
    check_q4_attention(out[:, good], ref[:, good.numpy()], A)


def test_small_query_rows_keep_their_own_precision(lib):
    # rows 2^-16 of those beside them, against keys large enough that their scores still are N(0, 1)
    L, H = 400, 2
    g = torch.Generator().manual_seed(4)
    K = torch.randn((1, L, H, 128), generator=g) * 2.0 ** 12
    V = torch.randn((1, L, H, 128), generator=g)
    q = torch.randn((1, 2, 8, 128), generator=g) * torch.tensor([2.0 ** 4, 2.0 ** -12])[None, :, None, None]
    q = q.bfloat16()
    table, total = table_for([L], 16, seed=2)
    kc, vc = lib.alloc_q4_pools(total, H, 128)
    lib.kv_block_append_q4(K.to(DEV), V.to(DEV), kc, vc, table.to(DEV), i32([L]))
    out = lib.spec_verify_attn_q4(q.to(DEV), kc, vc, table.to(DEV), i32([L]))
    ref, A = q4_reference(q, kc, vc, table, [L], 16)
    check_q4_attention(out[:, 1:], ref[:, 1:], A)
