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


@pytest.mark.parametrize("captured", [False, True])
def test_layers_of_all_kinds_share_a_workspace(lib, captured):
    # plain, windowed and 4-bit layers in turn over one workspace: grids of several waves (ordered work), contexts in
    # several splits (partials and a merge) and in one; bit-equal to a workspace each
    import workloads
    cfg = workloads.CONFIGS["tiny"].with_(kv_dtype="bf16", q_dtype="bf16", logit_dtype="bf16", B=64, H_q=16, H_kv=8,
                                          d_head=128, K=4, V=512, ctx=("uniform", (5, 3000)))
    a = {k: (t.to(DEV) if isinstance(t, torch.Tensor) else t) for k, t in
         {**workloads.make_attention_inputs(cfg, 0), **workloads.make_append_inputs(cfg, 0),
          **workloads.make_sampling_inputs(cfg, 0)}.items()}
    table = torch.full((64, 2048), -1, dtype=torch.int32, device=DEV)   # 32K tokens a sequence
    table[:, :a["block_table"].shape[1]] = a["block_table"]
    total = a["k_cache"].shape[0]
    g = torch.Generator(device=DEV).manual_seed(5)

    def bf16():
        return {n + "_cache": torch.randn(a[n + "_cache"].shape, generator=g, device=DEV).bfloat16() for n in "kv"}

    def fp8():
        return dict({n + "_cache": torch.randint(0, 120, a[n + "_cache"].shape, generator=g, device=DEV,
                                                 dtype=torch.uint8) for n in "kv"},
                    k_scale=torch.full((8,), 0.01, device=DEV), v_scale=torch.full((8,), 0.01, device=DEV))

    def q4():
        k, v = (p.to(DEV) for p in q4_pools(total, 8, 128, BS, seed=8, spread=False))
        return dict(k_cache=k, v_cache=v)

    kinds = [(bf16, 0, 0), (bf16, 1024, 4), (fp8, 0, 0), (q4, 0, 0), (bf16, 0, 0), (fp8, 500, 17), (bf16, 0, 0),
             (q4, 1024, 4), (bf16, 100, 0)]
    layers = []
    for k, (make, W, S) in enumerate(kinds):
        q = torch.randn(a["q"].shape, generator=g, device=DEV).bfloat16()
        layers.append(dict(make(), q=q, k_new=a["k_new"], v_new=a["v_new"], window=W, sinks=S))
    assert lib.attn_workspace_size(64, 5, 16, 8, 128, 2048) != lib.attn_window_workspace_size(64, 5, 16, 8, 128, 2048, 16,
                                                                                              1024, 4)
    sample = (a["target_logits"], a["draft_logits"], a["draft_tokens"], a["uniforms"])
    want = []
    for l in layers:
        m = lib.MultiLayerVerify([l], table, a["seq_lens"], *sample)
        m.run()
        torch.cuda.synchronize()
        assert int(m.status) == 0
        want.append(m.outs[0].clone())
    m = lib.MultiLayerVerify(layers, table, a["seq_lens"], *sample)
    if captured:
        m.capture()
    for _ in range(4):
        for o in m.outs:
            o.fill_(float("nan"))
        m.replay() if captured else m.run()
        torch.cuda.synchronize()
        assert int(m.status) == 0
        for o, w in zip(m.outs, want):
            assert torch.equal(o, w)


@pytest.mark.parametrize("B,n_new,H", [(96, 1, 16), (5, 4, 64), (1500, 1, 1)])
def test_latent_calls_of_other_lengths_share_a_workspace(lib, B, n_new, H):
    # one workspace, lengths that sort the other way round from call to call: bit-equal to a workspace each
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(n_new, 400 if B < 1000 else 40, (B,), generator=g).to(torch.int32)
    other = lens.max() + n_new - lens
    table, total = table_for([int(lens.max()) + n_new] * B, BS, seed=1)
    cache = torch.randn((total, BS, 576), generator=g).to(torch.bfloat16).to(DEV)
    q = torch.randn((B, n_new, H, 576), generator=g).to(torch.bfloat16).to(DEV)
    table, both = table.to(DEV), [lens.to(DEV), other.to(DEV)]
    want = []
    for L in both:
        want.append(lib.spec_verify_attn_mla(q, cache, table, L, 0.07))
        torch.cuda.synchronize()
    ws = lib.alloc_workspace(lib.mla_workspace_size(B, n_new, H, table.shape[1]), DEV)
    outs = [torch.empty_like(w) for w in want]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run():
        for _ in range(3):
            for L, o in zip(both, outs):
                lib.spec_verify_attn_mla(q, cache, table, L, 0.07, out=o, workspace=ws, status=st)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for go in (run, graph.replay):
        for o in outs:
            o.fill_(float("nan"))
        go()
        torch.cuda.synchronize()
        assert int(st) == 0
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
