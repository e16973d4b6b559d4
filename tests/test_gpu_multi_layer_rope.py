"""Rounds over layers of other heads and types, some of which rotate their rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("captured", [False, True])
def test_rotating_layers_unlike_the_first(lib, captured):
    B, n, d, V = 2, 3, 128, 1000
    lens = [150, 33]
    table = torch.arange(20, dtype=torch.int32).reshape(2, 10).to(DEV)
    g = torch.Generator(DEV).manual_seed(5)

    def rows(*shape, dtype):
        return torch.randn(shape, device=DEV, generator=g).to(dtype)

    def layer(H_q, H_kv, dtype, rope, strided=False, **over):
        if strided:   # queries and keys as heads of one projection, head by head
            qkv = rows(B, H_q + H_kv, n, d, dtype=dtype).transpose(1, 2)
            q, k = qkv[:, :, :H_q], qkv[:, :, H_q:]
        else:
            q, k = rows(B, n, H_q, d, dtype=dtype), rows(B, n, H_kv, d, dtype=dtype)
        if dtype == torch.float32:
            kc, vc = (rows(20, H_kv, 16, d, dtype=dtype) for _ in range(2))
        else:
            kc, vc = lib.alloc_q8_pools(20, H_kv, d)
            old = rows(B, 140, H_kv, d, dtype=dtype)
            lib.kv_block_append_q8(old[:, :30].contiguous(), old[:, :30].contiguous(), kc, vc, table, i32([30, 30]))
            lib.kv_block_append_q8(old[:1].contiguous(), old[:1].contiguous(), kc, vc, table[:1], i32([147]))
        return dict(q=q, k_new=k, v_new=rows(B, n, H_kv, d, dtype=dtype), k_cache=kc, v_cache=vc, rope=rope, **over)

    r, half = lib.Rope(128, theta=500000.0), lib.Rope(64, interleaved=True, offset=32)
    bf, f32 = torch.bfloat16, torch.float32
    layers = [layer(16, 4, f32, None), layer(16, 4, bf, r), layer(8, 2, bf, half, window=20, sinks=2), layer(16, 4, f32, half),
              layer(16, 4, bf, None), layer(8, 2, bf, r, strided=True), layer(16, 4, bf, half)]
    want = []
    for l in layers:   # each layer by its own calls, over copies of its pools
        q, k = l["q"], l["k_new"]
        if l["rope"] is not None:
            q, k = lib.spec_rope(q, k, l["rope"], seq_lens=i32(lens))
        kc, vc = l["k_cache"].clone(), l["v_cache"].clone()
        lib._append_any(k, l["v_new"], kc, vc, table, i32(lens), None, None, 16, None)
        want.append((lib._attn_any(q, kc, vc, table, i32(lens), None, None, None, l.get("window", 0), l.get("sinks", 0), 16, None,
                                   None, None), kc, vc))
    m = lib.MultiLayerVerify(layers, table, i32(lens), rows(B, n, V, dtype=f32), rows(B, n - 1, V, dtype=f32),
                             torch.randint(0, V, (B, n - 1), device=DEV, dtype=torch.int32, generator=g),
                             torch.rand((B, n, 2), device=DEV, generator=g))
    if captured:
        m.capture()
        m.replay()   # (the same rows into the same slots: the same pools)
    else:
        m.run()
    torch.cuda.synchronize()
    assert int(m.status) == 0
    for l, o, (ref, kc, vc) in zip(layers, m.outs, want):
        assert torch.equal(l["k_cache"], kc) and torch.equal(l["v_cache"], vc)
        assert torch.equal(o, ref)
