"""Calls of the library that follow one another on a stream, each reading or
overwriting what the one before it wrote or read: the same results as with a
synchronisation between them."""
import pytest
import torch

from q4_utils import q4_pools, table_for

pytestmark = pytest.mark.gpu
DEV = "cuda"
BS = 16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def bits(t):
    return t.view(torch.uint8)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype,target", [
    (torch.bfloat16, "q4"), (torch.float32, "q4"), (torch.bfloat16, "bf16"), (torch.float32, "f32"),
    (torch.bfloat16, "fp8"),
])
@pytest.mark.parametrize("B,H,rows", [(1, 2, 40), (4, 8, 333), (16, 8, 2048)])
def test_rows_read_back_move_to_another_cache(lib, dtype, target, captured, B, H, rows):
    # read back from one cache, appended to another, nothing between: bit-equal to the same with a synchronisation
    lens = [rows] * B
    table, total = table_for(lens, BS, seed=rows)
    table, L = table.to(DEV), i32(lens)
    src = [p.to(DEV) for p in q4_pools(total, H, 128, BS, seed=3, spread=False)]
    other = [p.to(DEV) for p in q4_pools(total, H, 128, BS, seed=7, spread=False)]
    start = torch.zeros_like(L)
    buf = [torch.empty((B, rows, H, 128), dtype=dtype, device=DEV) for _ in range(2)]
    scale = torch.full((H,), 0.02, device=DEV)

    def pools():
        if target == "q4":
            return lib.alloc_q4_pools(total, H, 128)
        t = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.uint8}[target]
        return tuple(torch.zeros((total, H, BS, 128), dtype=t, device=DEV) for _ in range(2))

    def move(pair, dst, sync=False):
        lib.kv_block_gather_q4(*pair, table, L, start, rows, 128, k_out=buf[0], v_out=buf[1])
        if sync:
            torch.cuda.synchronize()
        if target == "q4":
            lib.kv_block_append_q4(*buf, *dst, table, L)
        elif target == "fp8":
            lib.kv_block_append(*buf, *dst, table, L, scale, scale)
        else:
            lib.kv_block_append(*buf, *dst, table, L)

    want = []
    for pair in (src, other):
        dst = pools()
        move(pair, dst, sync=True)
        torch.cuda.synchronize()
        want.append(dst)
    assert not torch.equal(bits(want[0][0]), bits(want[1][0]))
    got = [pools(), pools()]

    def both():   # the second move overwrites the rows that the first one's append reads
        move(src, got[0])
        move(other, got[1])

    both()
    if captured:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            both()
    for _ in range(5):
        for t in buf:
            t.fill_(77)
        for pair in got:
            for t in pair:
                t.zero_()
        g.replay() if captured else both()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(bits(a[1]), bits(b[1]))
