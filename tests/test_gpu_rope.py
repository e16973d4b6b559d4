"""Rotary positions on the GPU against the fp64 oracle.

Bounds. A rotated element is scale (a cos - b sin), |a|, |b| <= M of its pair:
  * the angle: the fraction of a turn from 64-bit fixed point (2^-33 turns at
    32-bit positions), cut to 32 bits (2^-32 turns) and rounded to f32 as half
    turns within +-1 (2^-25): at most 2^-24.8 half turns in all, 2^-23 radians,
    which moves the element by at most 2^-23 (|a| + |b|) scale;
  * cosine and sine: 2 units in the last place of f32 (2^-22 of 1), times
    scale (2^-24): together 2^-21.7 (|a| + |b|) scale;
  * two products and a sum in f32: 2^-24 each of at most |a| + |b|, 2^-22.4;
  * the rounding to the output type: finfo.eps / 2 of the result.
So eps / 2 |ref| + 2^-20 (|a| + |b|) |scale|, the 2^-20 one binade above
2^-23 + 2^-21.7 + 2^-22.4 = 2^-20.7; for f16, 2^-25 besides (subnormals).
"""
import numpy as np
import pytest
import torch

from oracle import rope as orope

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def check(got, x, pos, rope):
    w = np.array(rope.inv_freq)
    x = x.detach().cpu().double().numpy()
    ref = orope.rotate(x, pos, w, rope.interleaved, rope.offset, rope.scale)
    other = orope.rotate(np.abs(x), np.zeros_like(pos), w, rope.interleaved, rope.offset)   # |a|, |b| in place
    r, o = 2 * len(w), rope.offset
    size = np.zeros_like(ref)
    part = other[..., o:o + r]
    if rope.interleaved:
        both = part[..., 0::2] + part[..., 1::2]
        size[..., o:o + r] = np.repeat(both, 2, axis=-1)
    else:
        both = part[..., :r // 2] + part[..., r // 2:]
        size[..., o:o + r] = np.concatenate((both, both), -1)
    err = np.abs(got.detach().cpu().double().numpy() - ref)
    eps = torch.finfo(got.dtype).eps / 2
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    assert (err <= eps * np.abs(ref) + 2.0 ** -20 * size * abs(rope.scale) + tiny * (size > 0)).all(), err.max()


SHAPES = [   # B, n, H_q, H_kv, d, r, offset
    (1, 1, 64, 8, 128, 128, 0), (3, 5, 32, 8, 128, 128, 0), (2, 3, 8, 1, 128, 64, 0), (2, 4, 128, 1, 576, 64, 512), (1, 7, 4, 4, 64, 32, 32),
    (2, 2, 3, 3, 80, 20, 10), (1, 3, 5, 2, 37, 6, 1), (2, 1, 1, 1, 2, 2, 0), (1, 2, 16, 2, 256, 256, 0), (1, 600, 2, 1, 16, 16, 0),
    (40, 33, 6, 2, 96, 48, 0), (1, 1, 3, 0, 128, 128, 0), (2, 3, 0, 5, 48, 16, 16), (1, 1100, 8, 2, 128, 126, 2),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,n,Hq,Hk,d,r,offset", SHAPES)
def test_rope(lib, B, n, Hq, Hk, d, r, offset, interleaved, dtype):
    rope = lib.Rope(r, theta=500000.0, interleaved=interleaved, offset=offset, scale=1.25)
    g = torch.Generator().manual_seed(d + n)
    q = torch.randn((B, n, Hq, d), generator=g).to(dtype) if Hq else None
    k = torch.randn((B, n, Hk, d), generator=g).to(dtype) if Hk else None
    lens = [n + (b * 7919) % 131072 for b in range(B)]
    pos = np.array([[L - n + j for j in range(n)] for L in lens])
    st = i32([0])
    qd, kd = (None if t is None else t.to(DEV) for t in (q, k))
    qo, ko = lib.spec_rope(qd, kd, rope, seq_lens=i32(lens), status=st)
    assert int(st) == 0
    for x, xd, out in ((q, qd, qo), (k, kd, ko)):
        if x is None:
            assert out is None
            continue
        check(out, x, pos, rope)
        assert torch.equal(xd.cpu(), x)   # the inputs stay
    # in place: the same bits
    lib.spec_rope(qd, kd, rope, seq_lens=i32(lens), q_out=qd, k_out=kd)
    for xd, out in ((qd, qo), (kd, ko)):
        assert xd is None or torch.equal(xd, out)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(lib, interleaved):
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 131071, 1048575, 16777217, 999999937]], dtype=torch.int32)
    for theta in (2.0, 10000.0, 1e6):
        rope = lib.Rope(128, theta=theta, interleaved=interleaved)
        q = torch.randn((1, 9, 4, 128), generator=torch.Generator().manual_seed(1))
        out, _ = lib.spec_rope(q.to(DEV), None, rope, positions=pos.to(DEV))
        check(out, q, pos.numpy().astype(np.int64), rope)
        assert torch.equal(out[:, 0].cpu(), q[:, 0])
        back, _ = lib.spec_rope(out, None, rope, positions=i32([[0, -1, 1, -(2 ** 31 - 1), -2 ** 31, -131071, -1048575, -16777217,
                                                                 -999999937]]))
        keep = [0, 1, 2, 3, 5, 6, 7, 8]   # (2^31 has no negative among 32 bits)
        assert (back[:, keep].cpu() - q[:, keep]).abs().max() < 2.0 ** -18 * 8


@pytest.mark.parametrize("scaling", [{"kind": "linear", "factor": 4.0},
                                     {"kind": "llama3", "factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0, "original_length": 8192},
                                     {"kind": "yarn", "factor": 32.0, "original_length": 4096}])
def test_stretched_contexts(lib, scaling):
    rope = lib.Rope(64, theta=10000.0, scaling=scaling, offset=8)
    q = torch.randn((2, 3, 4, 80), generator=torch.Generator().manual_seed(2)).bfloat16()
    out, _ = lib.spec_rope(q.to(DEV), None, rope, seq_lens=i32([100000, 5]))
    check(out, q, np.array([[99997, 99998, 99999], [2, 3, 4]]), rope)


def test_given_frequencies(lib):
    # any finite frequencies: above 2 pi, negative, zero
    w = [7.5, -0.3, 0.0, 100.25, 1e-9, 6.283185307179586]
    rope = lib.Rope(12, inv_freq=w)
    q = torch.randn((1, 4, 2, 12), generator=torch.Generator().manual_seed(3))
    out, _ = lib.spec_rope(q.to(DEV), None, rope, positions=i32([[0, 3, 1000, -77]]))
    check(out, q, np.array([[0, 3, 1000, -77]]), rope)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_heads_of_a_packed_projection(lib, interleaved, pad):
    # q, k as slices of [B, n, (Hq + 2 Hk) d + pad]; other strides and places (16-byte aligned or not) give the same bits
    B, n, Hq, Hk, d = 2, 3, 6, 2, 64
    rope = lib.Rope(48, interleaved=interleaved, offset=8)
    flat = torch.randn((B, n, (Hq + 2 * Hk) * d + pad), generator=torch.Generator().manual_seed(4)).bfloat16().to(DEV)
    q = flat[..., pad:pad + Hq * d].unflatten(-1, (Hq, d))
    k = flat[..., pad + Hq * d:pad + (Hq + Hk) * d].unflatten(-1, (Hk, d))
    assert not q.is_contiguous()
    lens = i32([900, 33])
    want = lib.spec_rope(q.contiguous(), k.contiguous(), rope, seq_lens=lens)
    got = lib.spec_rope(q, k, rope, seq_lens=lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0].is_contiguous()
    before = flat.clone()
    qt = torch.empty((B, Hq, n, d), dtype=q.dtype, device=DEV).transpose(1, 2)   # heads before positions
    lib.spec_rope(q, k, rope, seq_lens=lens, q_out=qt, k_out=k)   # (keys in place inside the projection)
    assert torch.equal(qt, want[0]) and torch.equal(k, want[1])
    before[..., pad + Hq * d:pad + (Hq + Hk) * d] = want[1].flatten(2)
    assert torch.equal(flat, before)
    one = flat[:, :1, :d].unflatten(-1, (1, d)).expand(B, 1, 5, d)   # one head read five times
    got, _ = lib.spec_rope(one, None, rope, seq_lens=lens)
    assert torch.equal(got, lib.spec_rope(one.contiguous(), None, rope, seq_lens=lens)[0])


def test_short_lengths_leave_the_rows(lib):
    q = torch.randn((4, 3, 2, 64), device=DEV)
    k = torch.randn((4, 3, 1, 64), device=DEV)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    rope, st = lib.Rope(64), i32([0])
    lib.spec_rope(q, k, rope, seq_lens=i32([3, 2, -1, 50]), q_out=qo, k_out=ko, status=st)
    assert int(st) == 1
    assert (qo[1:3] == 7).all() and (ko[1:3] == 7).all()
    want = lib.spec_rope(q[[0, 3]], k[[0, 3]], rope, seq_lens=i32([3, 50]))
    assert torch.equal(qo[[0, 3]], want[0]) and torch.equal(ko[[0, 3]], want[1])
    a, b = lib.spec_rope(q[:0], k[:0], rope, seq_lens=i32([]))
    assert a.shape == (0, 3, 2, 64) and b.shape == (0, 3, 1, 64)


def test_non_finite_elements_stay_in_their_pair(lib):
    rope = lib.Rope(64)
    q = torch.randn((1, 2, 2, 96), device=DEV)
    good, _ = lib.spec_rope(q, None, rope, seq_lens=i32([40]))
    q[0, 1, 1, 5], q[0, 0, 0, 70] = float("nan"), float("inf")   # a rotated dim; one that is copied
    out, _ = lib.spec_rope(q, None, rope, seq_lens=i32([40]))
    bad = torch.zeros_like(q, dtype=torch.bool)
    bad[0, 1, 1, 5] = bad[0, 1, 1, 37] = bad[0, 0, 0, 70] = True
    assert torch.equal(out[~bad], good[~bad]) and torch.isnan(out[0, 1, 1, [5, 37]]).all() and torch.isinf(out[0, 0, 0, 70])


def test_captured_and_replayed_with_other_lengths(lib):
    rope, lens = lib.Rope(128, theta=500000.0), i32([100, 900])
    q = torch.randn((2, 5, 8, 128), device=DEV).bfloat16()
    qo = torch.empty_like(q)
    lib.spec_rope(q, None, rope, seq_lens=lens, q_out=qo)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.spec_rope(q, None, rope, seq_lens=lens, q_out=qo)
    lens += 1000
    q.normal_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, lib.spec_rope(q, None, rope, seq_lens=lens)[0])


def test_scores_of_rotated_rows_depend_on_the_distance(lib):
    # through the cache: the same rows 100000 positions further on give the same attention, to the rows' rounding
    rope = lib.Rope(128, theta=500000.0)
    n, L = 3, 40
    k, v = (torch.randn((1, L, 2, 128), generator=torch.Generator().manual_seed(s)).to(DEV) for s in (1, 2))
    q = torch.randn((1, n, 8, 128), generator=torch.Generator().manual_seed(3)).to(DEV)
    outs = []
    for far in (0, 100000):
        pos = torch.arange(far, far + L, dtype=torch.int32, device=DEV)[None]
        qr, _ = lib.spec_rope(q, None, rope, positions=pos[:, -n:].contiguous())
        _, kr = lib.spec_rope(None, k, rope, positions=pos)
        kc, vc = (torch.zeros((3, 2, 16, 128), device=DEV) for _ in range(2))
        lib.kv_block_append(kr, v, kc, vc, i32([[0, 1, 2]]), i32([L]))
        outs.append(lib.spec_verify_attn(qr, kc, vc, i32([[0, 1, 2]]), i32([L])))
    # scores: sums of 128 products, each factor off by at most 2^-20 (|a| + |b|): 2^-19 sum |q||k| < 2^-19 2^9
    assert (outs[0] - outs[1]).abs().max() < 2.0 ** -10 * 8
