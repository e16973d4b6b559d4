"""Inputs, references and bounds of the 8-bit block-scaled cache tests.

Bounds, from the formulas (half a rounding step is finfo.eps / 2 relative):
  * append and read-back are exact but for the rounding to the output type,
    which is exact too where scales are powers of two;
  * attention with bf16 queries, bf16 outputs: the output's rounding, 2^-8
    |ref|; the weights' rounding, 2^-11 (f16) and then 2^-10 (three e5m2
    terms), so 3 x 2^-11 of at most A = max |v|; and the scores, a relative
    error of the weights of at most 2 x 2^-11 for the scores drawn here (the
    query's two e4m3 terms: 2^-17 of its largest element on each small one,
    below 2^-12 in the score for |q| <= 2^2 and |k| of 128 elements summing to
    2^8 after the scale 2^-3.5; the accumulation: |q| |k| summed over 128 terms
    is below 2^7 after the scale, times 2^-18), so 5 x 2^-11 A in all;
  * with fp32 queries the kernel is fp32 throughout: 2^-16 A.
Besides, the 2-norm of the error over the output's: 6e-3 (the output's
rounding alone is at most 2^-8 = 3.9e-3).
"""
import math

import numpy as np
import torch

from oracle import attention as oatt
from oracle import q8 as oq8
from q4_utils import table_for   # noqa: F401


def q8_pools(total, H_kv, d, bs, seed, spread=True):
    """A pair of pools (CPU uint8) that hold N(0, 1) rows, rows and blocks of other sizes among them."""
    out = []
    for s in (seed, seed + 1):
        x = torch.randn((total, H_kv, bs, d), generator=torch.Generator().manual_seed(s)).numpy()
        rng = np.random.default_rng(s)
        if spread:
            x = x * rng.choice([1.0, 1.0, 1.0, 2.0, 0.25, 1e-6], size=x.shape[:3])[..., None]
            x = x * rng.choice([1.0, 1.0, 0.125, 1e-9], size=x.shape[:2])[..., None, None]
            x[rng.random(x.shape[:3]) < 0.02] = 0.5
            x[rng.random(x.shape[:2]) < 0.02] = 0.0
        x = x.astype(np.float32)
        scales = np.empty((total, H_kv), np.float32)
        codes = np.empty(x.shape, np.uint8)
        for i in range(total):
            for g in range(H_kv):
                scales[i, g] = 2.0 ** oq8.exponent(float(np.abs(x[i, g]).max()))
        codes = oq8.encode(x, scales[..., None, None])
        out.append(torch.from_numpy(oq8.join(codes, scales)))
    return out


def q8_reference(q, k_cache, v_cache, table, lens, H_kv, bs, window=0, sinks=0, rows=None):
    """(fp64 outputs, A) of the listed sequences; others NaN."""
    qf = q.detach().cpu().double().numpy()
    B, n, _, d = qf.shape
    out = np.full(qf.shape, np.nan)
    A = 0.0
    kc, vc, tb = k_cache.cpu().numpy(), v_cache.cpu().numpy(), table.cpu().numpy()
    for b in (range(B) if rows is None else rows):
        L = int(lens[b])
        Kd, Vd = (oq8.dense(pool, tb[b], L, H_kv, d, bs) for pool in (kc, vc))
        vis = oatt.window_visibility(n, L, window, sinks) if window else None
        out[b] = oatt.dense_attention(qf[b], Kd, Vd, n, 1 / math.sqrt(d), visible=vis)
        seen = np.ones(L, bool) if vis is None else vis.any(axis=0)
        A = max(A, np.abs(Vd[seen]).max())
    return out, A


def check_q8_attention(out, ref, A, rows=None):
    got = out.detach().double().cpu().numpy()
    if rows is not None:
        got, ref = got[list(rows)], ref[list(rows)]
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    bound = 2.0 ** -8 * np.abs(ref) + 5 * 2.0 ** -11 * A if out.dtype == torch.bfloat16 else np.full_like(err, 2.0 ** -16 * A)
    assert (err <= bound).all(), "max abs error %.3g (A %.3g)" % (err.max(), A)
    rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert rel <= (6e-3 if out.dtype == torch.bfloat16 else 2e-5), "relative error %.3g" % rel
