"""Verify attention through a sliding window with sinks over f32, bf16 and e4m3
caches, against the fp64 oracle (bounds: the framework's per-type attention
bars, parity_utils.attn_tolerance)."""
import math

import numpy as np
import pytest
import torch

import workloads
from oracle import attention as oatt
from parity_utils import attn_tolerance

pytestmark = pytest.mark.gpu
DEV = "cuda"


def reference(cfg, a, window, sinks, rows=None):
    is8 = cfg.kv_dtype == "fp8_e4m3"
    q = a["q"].double().numpy()
    out = np.full(q.shape, np.nan)
    for b in (range(cfg.B) if rows is None else rows):
        L = int(a["seq_lens"][b])
        kv = [oatt.gather_dense(a[n + "_cache"], a["block_table"][b], L, cfg.block_size,
                                None if a[n + "_scale"] is None else a[n + "_scale"].numpy(), is8) for n in "kv"]
        vis = oatt.window_visibility(cfg.n_new, L, window, sinks) if window else None
        out[b] = oatt.dense_attention(q[b], *kv, cfg.n_new, 1 / math.sqrt(cfg.d_head), visible=vis)
    return out


def run(lib, cfg, a, window, sinks, **kw):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    g = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in a.items()}
    out = lib.spec_verify_attn_window(g["q"], g["k_cache"], g["v_cache"], g["block_table"], g["seq_lens"], window, sinks,
                                      k_scale=g["k_scale"], v_scale=g["v_scale"], block_size=cfg.block_size, status=st, **kw)
    assert int(st) == 0
    return out


def check(out, ref, cfg, rows=None):
    got = out.double().cpu().numpy()
    if rows is not None:
        got, ref = got[list(rows)], ref[list(rows)]
    assert np.isfinite(got).all()
    err = np.abs(got - ref).max()
    assert err <= attn_tolerance(cfg.kv_dtype), "max abs error %.3g" % err
    # weights and outputs in bf16 are each within 2^-8, e4m3's path adds the query's two-term split (2^-8)
    rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert rel <= {"f32": 2e-5, "bf16": 2.0 ** -7, "fp8_e4m3": 3 * 2.0 ** -8}[cfg.kv_dtype], rel


SHAPES = [
    ("f32", dict(H_q=4, H_kv=2, d_head=64, K=4, ctx=(40, 64, 5, 300))),
    ("f32", dict(H_q=4, H_kv=1, d_head=96, K=0, ctx=(1, 77), block_size=8)),
    ("bf16", dict(H_q=8, H_kv=2, d_head=64, K=2, ctx=(90, 3, 200))),
    ("bf16", dict(H_q=8, H_kv=8, d_head=128, K=0, ctx=(1, 250, 64))),
    ("bf16", dict(H_q=16, H_kv=2, d_head=128, K=4, ctx=(5, 700, 333))),
    ("bf16", dict(H_q=16, H_kv=1, d_head=128, K=7, ctx=(1200, 8))),
    ("fp8_e4m3", dict(H_q=8, H_kv=2, d_head=64, K=4, ctx=(77, 250))),
    ("fp8_e4m3", dict(H_q=8, H_kv=2, d_head=128, K=8, ctx=(9, 517, 129))),
    ("fp8_e4m3", dict(H_q=32, H_kv=2, d_head=128, K=5, ctx=(700, 21))),
]
WINDOWS = [(0, 0), (1, 0), (4, 1), (16, 16), (50, 17), (64, 64), (129, 0), (200, 3), (33, 5000), (2 ** 31 - 1, 3)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("kv,over", SHAPES, ids=["%s-%d" % (s[0], i) for i, s in enumerate(SHAPES)])
def test_window(lib, kv, over, window, sinks):
    over = dict(over)
    ctx = over.pop("ctx")
    cfg = workloads.CONFIGS["tiny"].with_(kv_dtype=kv, q_dtype="f32" if kv == "f32" else "bf16", B=len(ctx),
                                          ctx=("fixed", ctx), **over)
    a = workloads.make_attention_inputs(cfg, seed=3)
    check(run(lib, cfg, a, window, sinks), reference(cfg, a, window, sinks), cfg)


@pytest.mark.parametrize("kv", ["f32", "bf16", "fp8_e4m3"])
def test_a_window_over_everything_is_plain_attention(lib, kv):
    cfg = workloads.CONFIGS["tiny"].with_(kv_dtype=kv, q_dtype="f32" if kv == "f32" else "bf16", d_head=128,
                                          ctx=("fixed", (250, 77)))
    a = workloads.make_attention_inputs(cfg, seed=5)
    g = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in a.items()}
    plain = lib.spec_verify_attn(g["q"], g["k_cache"], g["v_cache"], g["block_table"], g["seq_lens"], None, g["k_scale"],
                                 g["v_scale"])
    for W, S in ((0, 0), (256, 0), (10 ** 6, 50)):
        assert torch.equal(plain, run(lib, cfg, a, W, S))


@pytest.mark.parametrize("window,sinks", [(1024, 4), (100, 0), (2500, 33)])
@pytest.mark.parametrize("kv,B,H_q,K,lo,hi", [("bf16", 40, 64, 4, 5, 6000), ("fp8_e4m3", 90, 32, 8, 9, 2000),
                                              ("bf16", 1, 64, 7, 40000, 40000), ("fp8_e4m3", 2, 32, 0, 9000, 30000)])
def test_window_large(lib, kv, B, H_q, K, lo, hi, window, sinks):
    cfg = workloads.CONFIGS["tiny"].with_(kv_dtype=kv, q_dtype="bf16", B=B, H_q=H_q, H_kv=8, d_head=128, K=K,
                                          ctx=("uniform", (lo, hi)))
    a = workloads.make_attention_inputs(cfg, seed=1)
    rows = sorted({0, B // 2, B - 1})
    check(run(lib, cfg, a, window, sinks), reference(cfg, a, window, sinks, rows), cfg, rows)


@pytest.mark.parametrize("kv", ["f32", "bf16", "fp8_e4m3"])
def test_window_reads_no_other_pages(lib, kv):
    # released pages are -1 in the table; hidden keys of the pages that are read hold NaN (e4m3: its NaN code)
    W, S = 50, 18
    cfg = workloads.CONFIGS["tiny"].with_(kv_dtype=kv, q_dtype="f32" if kv == "f32" else "bf16", d_head=128,
                                          ctx=("fixed", (500, 300)))
    a = workloads.make_attention_inputs(cfg, seed=3)
    ref = reference(cfg, a, W, S)
    for b, L in enumerate((500, 300)):
        t = np.arange(L)
        hidden = (t >= S) & (t <= L - cfg.n_new - W)
        for blk in range(-(-L // 16)):
            here = hidden[blk * 16:(blk + 1) * 16]
            for n in ("k_cache", "v_cache"):
                a[n][int(a["block_table"][b, blk]), :, np.flatnonzero(here)] = 0x7F if kv == "fp8_e4m3" else float("nan")
            if here.all():
                a["block_table"][b, blk] = -1
    check(run(lib, cfg, a, W, S), ref, cfg)


def test_window_strided_pool_and_explicit_buffers(lib):
    # one layer of a pool [blocks][slots][layers][H_kv][d]; outputs and workspace of the caller's
    cfg = workloads.CONFIGS["tiny"].with_(kv_dtype="bf16", q_dtype="bf16", d_head=128, ctx=("fixed", (250, 77)))
    a = workloads.make_attention_inputs(cfg, seed=5)
    want = run(lib, cfg, a, 60, 5)
    nb, H, bs, d = a["k_cache"].shape
    big = [torch.zeros(nb, bs, 3, H, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for t, n in zip(big, ("k_cache", "v_cache")):
        t[:, :, 1] = a[n].to(DEV).transpose(1, 2)
    layout = (bs * 3 * H * d, d, 3 * H * d)
    ws = lib.alloc_workspace(lib.attn_window_workspace_size(2, cfg.n_new, cfg.H_q, H, d, a["block_table"].shape[1],
                                                            16, 60, 5), DEV)
    out = torch.empty_like(want)
    got = lib.spec_verify_attn_window(a["q"].to(DEV), big[0].view(-1)[H * d:], big[1].view(-1)[H * d:],
                                      a["block_table"].to(DEV), a["seq_lens"].to(DEV), 60, 5, layout=layout, num_blocks=nb,
                                      H_kv=H, out=out, workspace=ws)
    assert got is out and torch.equal(out, want)


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_window_bad_lengths_and_blocks(lib, kv):
    cfg = workloads.CONFIGS["tiny"].with_(kv_dtype=kv, q_dtype="bf16", d_head=128, B=3, ctx=("fixed", (200, 200, 200)))
    a = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in workloads.make_attention_inputs(cfg, 3).items()}
    good = lib.spec_verify_attn_window(a["q"], a["k_cache"], a["v_cache"], a["block_table"], a["seq_lens"], 40, 4,
                                       k_scale=a["k_scale"], v_scale=a["v_scale"])
    a["seq_lens"][0] = 2
    a["block_table"][1, -1] = 10 ** 6
    out = torch.full_like(good, 7.0)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.spec_verify_attn_window(a["q"], a["k_cache"], a["v_cache"], a["block_table"], a["seq_lens"], 40, 4, out=out,
                                k_scale=a["k_scale"], v_scale=a["v_scale"], status=st)
    assert int(st) == 1 | 2
    assert (out[0] == 7).all() and torch.equal(out[2], good[2])


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_window_graph_replay(lib, kv):
    cfg = workloads.CONFIGS["tiny"].with_(kv_dtype=kv, q_dtype="bf16", d_head=128, H_q=16, H_kv=2, ctx=("fixed", (900, 77)))
    a = workloads.make_attention_inputs(cfg, seed=5)
    g = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in a.items()}
    out = torch.empty_like(g["q"])
    ws = lib.alloc_workspace(lib.attn_window_workspace_size(2, cfg.n_new, 16, 2, 128, a["block_table"].shape[1], 16, 300, 9), DEV)

    def one():
        lib.spec_verify_attn_window(g["q"], g["k_cache"], g["v_cache"], g["block_table"], g["seq_lens"], 300, 9,
                                    k_scale=g["k_scale"], v_scale=g["v_scale"], out=out, workspace=ws)

    one()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    a["q"] = torch.randn(a["q"].shape, generator=torch.Generator().manual_seed(1)).bfloat16()
    a["seq_lens"] = torch.tensor([400, 60], dtype=torch.int32)
    g["q"].copy_(a["q"])
    g["seq_lens"].copy_(a["seq_lens"])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    check(out, reference(cfg, a, 300, 9), cfg)
