"""Inputs, references and bounds of the 4-bit cache and window tests.

Bounds, from the formulas (half a rounding step is finfo.eps / 2 relative):
  * read-back: one rounding to the output type of code * s + m, itself one
    fp32 fma: 2^-8 |v| for bf16, 2^-23 (code s + |m|) for f32;
  * attention over 4-bit pools with bf16 outputs: the output's rounding,
    2^-8 |ref|; the weights' rounding to f16, 2^-11 of at most A = max (15 s +
    |m|) over the values; and the scores' fp32 accumulation, a relative error
    of the weights of at most 2 x 2^-11 for the scores drawn here (|q| |k|
    summed over 128 terms is below 2^7 after the scale, times 2^-18), so
    3 x 2^-11 A < 2^-9 A in all;
  * with fp32 queries the kernel is fp32 throughout: 2^-16 A.
Besides, the 2-norm of the error over the output's: 6e-3 (the output's
rounding alone is at most 2^-8 = 3.9e-3).
"""
import math

import numpy as np
import torch

from oracle import attention as oatt
from oracle import q4 as oq4


def table_for(lens, bs, seed, spare=3, max_blocks=None):
    nblk = [(L + bs - 1) // bs for L in lens]
    total = sum(nblk) + spare
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lens), max_blocks or max(max(nblk), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(nblk):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total


def q4_pools(total, H_kv, d, bs, seed, spread=True):
    """A pair of pools (CPU uint8) that hold N(0, 1) rows, rows of other sizes among them."""
    out = []
    for kind, s in (("k", seed), ("v", seed + 1)):
        x = torch.randn((total, H_kv, bs, d), generator=torch.Generator().manual_seed(s)).numpy()
        if spread:   # some rows larger, some tiny, some constant
            rng = np.random.default_rng(s)
            f = rng.choice([1.0, 1.0, 1.0, 2.0, 0.25, 1e-6], size=x.shape[:3])
            x = x * f[..., None]
            x[rng.random(x.shape[:3]) < 0.02] = 0.5
        out.append(torch.from_numpy(oq4.pack(kind, *oq4.quantize(x.astype(np.float32)))))
    return out


def q4_reference(q, k_cache, v_cache, table, lens, bs, window=0, sinks=0, rows=None):
    """(fp64 outputs, A) of the listed sequences; others NaN."""
    qf = q.detach().cpu().double().numpy()
    B, n, _, d = qf.shape
    out = np.full(qf.shape, np.nan)
    A = 0.0
    kc, vc, tb = k_cache.cpu().numpy(), v_cache.cpu().numpy(), table.cpu().numpy()
    for b in (range(B) if rows is None else rows):
        L = int(lens[b])
        Kd, Vd = (oq4.dense(kind, pool, tb[b], L, d, bs) for kind, pool in (("k", kc), ("v", vc)))
        vis = oatt.window_visibility(n, L, window, sinks) if window else None
        out[b] = oatt.dense_attention(qf[b], Kd, Vd, n, 1 / math.sqrt(d), visible=vis)
        seen = np.ones(L, bool) if vis is None else vis.any(axis=0)
        blk = np.maximum(tb[b], 0)[: (L + bs - 1) // bs]
        _, s, m = oq4.unpack("v", vc[blk], d, bs)
        top = (15 * s.astype(float) + np.abs(m.astype(float))).max(axis=1).reshape(-1)[:L]
        A = max(A, top[seen].max())
    return out, A


def check_q4_attention(out, ref, A, rows=None):
    got = out.detach().double().cpu().numpy()
    if rows is not None:
        got, ref = got[list(rows)], ref[list(rows)]
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * A if out.dtype == torch.bfloat16 else np.full_like(err, 2.0 ** -16 * A)
    assert (err <= bound).all(), "max abs error %.3g (A %.3g)" % (err.max(), A)
    rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert rel <= (6e-3 if out.dtype == torch.bfloat16 else 2e-5), "relative error %.3g" % rel
