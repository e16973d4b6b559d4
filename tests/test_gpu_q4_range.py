"""Verify attention over 4-bit pools where weights and queries span a wide
range: one key that holds most of a long row's weight, and query rows of very
different sizes side by side."""
import math

import pytest
import torch

from q4_utils import check_q4_attention, q4_reference

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
