"""The 8-bit cache and rotary positions where their calls meet others: waits
that run out, layers of several kinds over one
workspace, rows too many for the append's registers."""
import numpy as np
import pytest
import torch

from oracle import q8 as oq8
from q8_utils import check_q8_attention, q8_pools, q8_reference, table_for
from test_gpu_rope import check as check_rope

pytestmark = pytest.mark.gpu
DEV = "cuda"


def status0():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def pools_of(lib, kind, lens, H, seed):
    """Filled pools of a kind and the table over them, on the GPU."""
    table, total = table_for(lens, 16, seed=seed)
    table = table.to(DEV)
    if kind == "q8":
        kc, vc = (p.to(DEV) for p in q8_pools(total, H, 128, 16, seed=seed, spread=False))
    else:
        kc, vc = lib.alloc_q4_pools(total, H, 128)
        n = max(lens)
        k, v = (torch.randn((len(lens), n, H, 128), device=DEV, generator=torch.Generator(DEV).manual_seed(seed + i)) for i in range(2))
        for b, L in enumerate(lens):
            lib.kv_block_append_q4(k[b:b + 1, :L].contiguous(), v[b:b + 1, :L].contiguous(), kc, vc, table[b:b + 1].contiguous(), i32([L]))
    return kc, vc, table


@pytest.mark.parametrize("H_q,H_kv,n", [(8, 2, 1), (64, 8, 3), (64, 8, 5), (64, 8, 6), (64, 8, 8)])
def test_waits_that_run_out(lib, H_q, H_kv, n):
    lens = [700, 333, 40]
    table, total = table_for(lens, 16, seed=3)
    kc, vc = q8_pools(total, H_kv, 128, 16, seed=9)
    q = torch.randn((3, n, H_q, 128), generator=torch.Generator().manual_seed(2)).bfloat16()
    args = (q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), i32(lens))
    st = status0()
    try:
        lib.test_hooks(2_000_000, lib.SV_TEST_WITHHOLD_COPIES)
        lib.spec_verify_attn_q8(*args, status=st)
        torch.cuda.synchronize()
    finally:
        lib.test_hooks(0, 0)
    assert int(st) & lib.SV_DEV_TIMEOUT
    st.zero_()
    out = lib.spec_verify_attn_q8(*args, status=st)
    assert int(st) == 0
    check_q8_attention(out, *q8_reference(q, kc, vc, table, lens, H_kv, 16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("where", [0, 130, 1000])
def test_append_of_rows_beyond_the_registers_leaves_nan_out(lib, dtype, where):
    # a block of 64 slots of 256: eight batches of a warp; the NaN lies in one of them
    d, bs, H, lens = 256, 64, 2, (64, 130)
    table, total = table_for(lens, bs, seed=1)
    kc, vc = q8_pools(total, H, d, bs, seed=3)
    k, v = (torch.randn((2, 64, H, d), generator=torch.Generator().manual_seed(i)).to(dtype) for i in range(2))
    k.view(-1)[where * 16:where * 16 + 3] = float("nan")
    v[1, :, 1] = float("nan")
    kd, vd = kc.to(DEV), vc.to(DEV)
    lib.kv_block_append_q8(k.to(DEV), v.to(DEV), kd, vd, table.to(DEV), i32(lens), block_size=bs)
    want = oq8.append(kc.numpy(), vc.numpy(), k.float().numpy(), v.float().numpy(), table.numpy(), lens, bs)
    for got, ref in zip((kd, vd), want):
        assert np.array_equal(got.cpu().numpy(), ref)


def test_layers_of_all_kinds_share_a_workspace(lib):
    lens, H = [500, 64, 1203], 2
    q = torch.randn((3, 4, 16, 128), device=DEV, generator=torch.Generator(DEV).manual_seed(8)).bfloat16()
    q8 = pools_of(lib, "q8", lens, H, seed=1)
    q4 = pools_of(lib, "q4", lens, H, seed=2)
    t = table_for(lens, 16, seed=3)[0].to(DEV)
    bf = tuple(torch.randn((int(t.max()) + 1, H, 16, 128), device=DEV).bfloat16() for _ in range(2))
    mb = t.shape[1]
    size = max(lib.attn_q8_workspace_size(3, 4, 16, H, 128, mb), lib.attn_q4_workspace_size(3, 4, 16, H, 128, mb),
               lib.attn_workspace_size(3, 4, 16, H, 128, mb))
    ws = lib.alloc_workspace(size, DEV)
    ws.fill_(255)
    L = i32(lens)

    def layers(w):
        return [lib.spec_verify_attn_q8(q, *q8, L, workspace=w), lib.spec_verify_attn(q, *bf, t, L, workspace=w),
                lib.spec_verify_attn_q8(q[:, :1].contiguous(), *q8, L, workspace=w), lib.spec_verify_attn_q4(q, *q4, L, workspace=w),
                lib.spec_verify_attn_q8(q, *q8, L, window=100, sinks=3, workspace=w)]
    alone = layers(None)
    for _ in range(20):
        for a, b in zip(layers(ws), alone):
            assert torch.equal(a, b)


# Heads in many turns, pieces beyond a CTA's threads, an odd number of vectors that stay.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,n,Hq,Hk,d,r,offset", [
    (1, 2, 300, 5, 40, 16, 0), (2, 3, 7, 3, 601, 32, 1), (2, 2, 130, 1, 40, 16, 24), (700, 1, 33, 2, 128, 128, 0), (1, 1, 2, 1, 2056, 256, 8),
    (620, 1, 1, 1, 1032, 250, 3),
])
def test_rope_of_other_shapes(lib, B, n, Hq, Hk, d, r, offset, interleaved, dtype):
    g = torch.Generator().manual_seed(d + B)
    q, k = (torch.randn((B, n, H, d), generator=g).to(dtype).to(DEV) for H in (Hq, Hk))
    lens = torch.randint(n, 5000, (B,), generator=g, dtype=torch.int32)
    rope = lib.Rope(r, theta=10000.0, interleaved=interleaved, offset=offset)
    pos = lens[:, None].numpy() - n + np.arange(n)
    qo, ko = lib.spec_rope(q, k, rope, seq_lens=lens.to(DEV))
    check_rope(qo, q, pos, rope)
    check_rope(ko, k, pos, rope)
    # queries in place, keys not
    q2 = q.clone()
    same, ko2 = lib.spec_rope(q2, k, rope, seq_lens=lens.to(DEV), q_out=q2)
    assert same is q2 and torch.equal(q2, qo) and torch.equal(ko2, ko)


def test_rope_outputs_side_by_side(lib):
    # rows of a head next to one another, heads further apart: not in the order of the dims, but apart
    q = torch.randn((3, 2, 5, 64), device=DEV).bfloat16()
    out = torch.zeros((3, 5, 2, 64), device=DEV, dtype=torch.bfloat16).transpose(1, 2)
    rope = lib.Rope(64)
    lens = i32([9, 2, 300])
    want, _ = lib.spec_rope(q, None, rope, seq_lens=lens)
    got, _ = lib.spec_rope(q, None, rope, seq_lens=lens, q_out=out)
    assert got is out and torch.equal(out, want)


def test_rope_of_no_heads(lib):
    rope, lens = lib.Rope(64), i32([9, 300])
    k = torch.randn((2, 3, 4, 64), device=DEV).bfloat16()
    want = lib.spec_rope(None, k, rope, seq_lens=lens)[1]
    none = k[:, :, :0].contiguous()
    q, got = lib.spec_rope(none, k, rope, seq_lens=lens)
    assert q.shape == none.shape and torch.equal(got, want)
    got, q = lib.spec_rope(k, none, rope, seq_lens=lens)
    assert q.shape == none.shape and torch.equal(got, want)
    q, got = lib.spec_rope(none, none, rope, seq_lens=lens)
    assert q.shape == none.shape == got.shape
