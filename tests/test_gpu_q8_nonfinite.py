"""Verify attention over 8-bit block-scaled pools with infinite and NaN query elements: the row
that holds one comes out as NaN, as the formula has it (a score of +Inf makes Inf - Inf in the
softmax), and the other rows keep their bits."""
import pytest
import torch

from q8_utils import q8_pools, table_for

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = float("inf"), float("nan")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 3)])
@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 128), (torch.bfloat16, 64)])
@pytest.mark.parametrize("H_q,H_kv,n,lens", [(8, 2, 3, (200, 5)), (64, 8, 5, (700,)), (64, 8, 8, (1500, 9)), (8, 8, 1, (3000, 40))])
def test_rows_that_hold_an_infinity_are_nan(lib, H_q, H_kv, n, lens, dtype, d, window, sinks):
    table, total = table_for(lens, 16, seed=4)
    kc, vc = (p.to(DEV) for p in q8_pools(total, H_kv, d, 16, seed=6, spread=False))
    q = torch.randn((len(lens), n, H_q, d), generator=torch.Generator().manual_seed(n)).to(dtype).to(DEV)
    good = lib.spec_verify_attn_q8(q, kc, vc, table.to(DEV), i32(lens), window=window, sinks=sinks)
    assert torch.isfinite(good).all()
    bad = torch.zeros(len(lens), n, H_q, dtype=torch.bool)
    last = 0 if lens[-1] < 40 else len(lens) - 1   # (a sequence with codes of both signs in every dim: some score is +Inf)
    for b, j, h, c, x in ((0, 0, 0, 0, INF), (0, n - 1, 5, d - 1, -INF), (0, n // 2, 3, 37, NAN), (last, n - 1, 7, 17, INF)):
        q[b, j, h, c] = x
        bad[b, j, h] = True
    q[0, 0, 0, 5] = -INF   # (two in one row)
    st = i32([0])
    out = lib.spec_verify_attn_q8(q, kc, vc, table.to(DEV), i32(lens), window=window, sinks=sinks, status=st)
    assert int(st) == 0
    assert torch.isnan(out[bad.to(DEV)]).all()
    assert torch.equal(out[~bad.to(DEV)], good[~bad.to(DEV)])


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_an_infinity_against_codes_of_one_sign(lib, sign):
    # every score of the row is +Inf, or every one -Inf: no weight is defined either way
    H, L = 2, 300
    K = torch.rand((1, L, H, 128), generator=torch.Generator().manual_seed(1)) + 0.5
    V = torch.randn((1, L, H, 128), generator=torch.Generator().manual_seed(2))
    table, total = table_for([L], 16, seed=2)
    kc, vc = lib.alloc_q8_pools(total, H, 128)
    lib.kv_block_append_q8(K.to(DEV), V.to(DEV), kc, vc, table.to(DEV), i32([L]))
    q = torch.randn((1, 2, 8, 128), generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    q[0, 1, 6, 9] = sign * INF
    out = lib.spec_verify_attn_q8(q, kc, vc, table.to(DEV), i32([L]))
    bad = torch.zeros(1, 2, 8, dtype=torch.bool, device=DEV)
    bad[0, 1, 6] = True
    assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()
