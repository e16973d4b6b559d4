"""The oracle of rotary positions against the latent oracle's rotation, complex
numbers, and closed forms; and the library's host-side frequencies."""
import ctypes
import math

import numpy as np
import pytest

import speculative_verify_paged_gb300 as sv
from oracle import mla as omla
from oracle import rope


@pytest.fixture(scope="module", autouse=True)
def lib():
    sv.build()
    return sv.load_library()


def test_interleaved_is_the_latent_rotation():
    x = np.random.default_rng(0).standard_normal((1, 7, 3, 64))
    pos = np.arange(100, 107)[None]
    got = rope.rotate(x, pos, rope.frequencies(64), interleaved=True)
    want = np.moveaxis(omla.rope(np.moveaxis(x, 1, 2), pos[0]), 2, 1)
    assert np.allclose(got, want, rtol=0, atol=1e-12)


def test_half_is_interleaved_in_another_order():
    x = np.random.default_rng(1).standard_normal((2, 3, 2, 20))
    pos = np.array([[5, 9, 1], [0, 70000, -3]])
    w = rope.frequencies(20, 500000.0)
    order = np.stack((np.arange(10), np.arange(10, 20)), 1).reshape(-1)   # i, i + 10, i + 1, ...
    inter = rope.rotate(x[..., order], pos, w, interleaved=True, scale=1.25)
    assert np.allclose(rope.rotate(x, pos, w, scale=1.25)[..., order], inter, rtol=0, atol=1e-12)


def test_rotation_by_complex_numbers_and_back():
    x = np.random.default_rng(2).standard_normal((1, 4, 1, 40))
    pos = np.array([[0, 1, 2, 131071]])
    w = rope.frequencies(16)
    y = rope.rotate(x, pos, w, interleaved=True, offset=6)
    z = (x[..., 6:22:2] + 1j * x[..., 7:22:2]) * np.exp(1j * pos[0][:, None, None] * w)
    assert np.allclose(y[..., 6:22:2], z.real, atol=1e-12) and np.allclose(y[..., 7:22:2], z.imag, atol=1e-12)
    assert np.array_equal(y[..., :6], x[..., :6]) and np.array_equal(y[..., 22:], x[..., 22:])
    assert np.array_equal(y[:, 0], x[:, 0])
    assert np.allclose(rope.rotate(y, -pos, w, interleaved=True, offset=6), x, atol=1e-12)


def test_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((1, 1, 1, 32)), rng.standard_normal((1, 1, 1, 32))
    w = rope.frequencies(32)
    dots = [float((rope.rotate(q, [[p + 7]], w) * rope.rotate(k, [[p]], w)).sum()) for p in (0, 5, 1000)]
    assert np.allclose(dots, dots[0], atol=1e-10)


@pytest.mark.parametrize("r,theta", [(128, 500000.0), (64, 10000.0), (6, 10000.0), (256, 1e6), (2, 2.0)])
def test_library_frequencies(r, theta):
    w = rope.frequencies(r, theta)
    assert np.allclose(sv.Rope(r, theta).inv_freq, w, rtol=1e-14)
    assert np.allclose(sv.Rope(r, theta, scaling={"kind": "linear", "factor": 4}).inv_freq, rope.linear(w, 4.0), rtol=1e-14)
    s = {"kind": "llama3", "factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0, "original_length": 8192}
    assert np.allclose(sv.Rope(r, theta, scaling=s).inv_freq, rope.llama3(w, 8.0, 1.0, 4.0, 8192), rtol=1e-12)
    for factor in (32.0, 0.5):
        h = sv.Rope(r, theta, scaling={"kind": "yarn", "factor": factor, "original_length": 4096}, scale=2.0)
        want, m = rope.yarn(w, theta, factor, 32.0, 1.0, 4096)
        assert np.allclose(h.inv_freq, want, rtol=1e-12) and math.isclose(h.scale, 2 * m, rel_tol=1e-6)
    h = sv.Rope(r, theta, scaling={"kind": "yarn", "factor": 4, "original_length": 4096, "attention_factor": 0.75, "beta_fast": 20})
    assert np.allclose(h.inv_freq, rope.yarn(w, theta, 4.0, 20.0, 1.0, 4096)[0], rtol=1e-12) and h.scale == 0.75


def test_llama3_keeps_short_and_divides_long_wavelengths():
    w = rope.frequencies(128, 500000.0)
    out = np.array(sv.Rope(128, 500000.0, scaling={"kind": "llama3", "factor": 8, "low_freq_factor": 1, "high_freq_factor": 4,
                                                   "original_length": 8192}).inv_freq)
    length = 2 * np.pi / w
    assert np.array_equal(out[length < 2048], w[length < 2048])
    assert np.allclose(out[length > 8192], w[length > 8192] / 8, rtol=1e-14)
    assert (np.diff(out) < 0).all()


def test_rope_refusals(lib):
    for r in (0, 3, -2, 258):
        with pytest.raises(sv.SpecVerifyError):
            sv.Rope(r)
    for theta in (1.0, 0.0, float("inf"), float("nan")):
        with pytest.raises(sv.SpecVerifyError):
            sv.Rope(64, theta)
    with pytest.raises(ValueError, match="kinds"):
        sv.Rope(64, scaling={"kind": "cubic", "factor": 2})
    with pytest.raises(ValueError, match="takes"):
        sv.Rope(64, scaling={"kind": "yarn", "factor": 2})
    with pytest.raises(ValueError, match="takes"):
        sv.Rope(64, scaling={"kind": "linear", "factor": 2, "beta_fast": 1})
    for bad in ({"kind": "linear", "factor": 0.0}, {"kind": "linear", "factor": float("nan")},
                {"kind": "llama3", "factor": 8, "low_freq_factor": 4, "high_freq_factor": 4, "original_length": 8192},
                {"kind": "yarn", "factor": 2, "original_length": -1}):
        with pytest.raises(sv.SpecVerifyError):
            sv.Rope(64, scaling=bad)
    with pytest.raises(ValueError, match="attention_factor"):
        sv.Rope(64, scaling={"kind": "yarn", "factor": 2, "original_length": 4096, "attention_factor": 0})
    with pytest.raises(ValueError, match="inv_freq"):
        sv.Rope(64, inv_freq=[1.0] * 31)
    with pytest.raises(ValueError, match="inv_freq"):
        sv.Rope(4, inv_freq=[1.0, float("nan")])
    with pytest.raises(ValueError, match="offset"):
        sv.Rope(64, offset=-1)
    with pytest.raises(ValueError, match="scale"):
        sv.Rope(64, scale=float("inf"))


FAKE, NULL = ctypes.c_void_p(0x1000), None
OTHER = ctypes.c_void_p(0x20000)


def call(lib, r, q=FAKE, qo=OTHER, k=FAKE, ko=OTHER, dt=1, pos=NULL, lens=FAKE, B=2, n=3, Hq=4, Hk=2, d=64, rows=(None,) * 4):
    return lib.spec_rope(q, qo, k, ko, dt, *[ctypes.byref(sv._RopeRows(*x)) if x else None for x in rows], r._ref if r else None,
                         pos, lens, B, n, Hq, Hk, d, NULL, NULL)


def test_call_refusals(lib):
    r = sv.Rope(64)
    for over in (dict(q=NULL), dict(qo=NULL), dict(k=NULL), dict(ko=NULL), dict(lens=NULL), dict(B=-1), dict(n=0), dict(d=1),
                 dict(Hq=0, Hk=0), dict(Hq=-1), dict(d=62), dict(rows=((0, 0, -1), None, None, None)),
                 dict(rows=(None, (12, 4, 63), None, None)), dict(rows=(None, None, None, (384, 63, 128))),
                 dict(qo=FAKE, rows=((1024, 256, 64), (2048, 256, 64), None, None))):
        assert call(lib, r, **over) == 1, over
    assert call(lib, None) == 1
    assert call(lib, r, dt=3) == 2 and call(lib, r, d=70000) == 2 and call(lib, r, Hq=65535) == 2
    assert call(lib, r, B=1 << 20, n=1 << 12) == 2
    assert call(lib, sv.Rope(32, offset=33)) == 1
    assert call(lib, r, B=0) == 0 and call(lib, r, B=0, q=NULL, qo=NULL, Hq=0) == 0
    bad = sv.Rope(64)
    bad._c.rotary_dim = 63
    assert call(lib, bad) == 1
    bad = sv.Rope(64)
    bad._c.inv_freq[5] = float("inf")
    assert call(lib, bad) == 1
    bad = sv.Rope(64)
    bad._c.scale = float("nan")
    assert call(lib, bad) == 1


def test_binding_refusals():
    import torch
    q, k = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    lens, pos = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    r = sv.Rope(64)
    with pytest.raises(TypeError, match="Rope"):
        sv.spec_rope(q, k, None, seq_lens=lens)
    for args, over, msg in (((q, k), {}, "needed"), ((q, k.float()), dict(seq_lens=lens), "one dtype"),
                            ((None, None), dict(seq_lens=lens), "must be"), ((q[0], k), dict(seq_lens=lens), "must be"),
                            ((q, k[:, :2]), dict(seq_lens=lens), "must be"), ((q, k), dict(seq_lens=lens.long()), "int32"),
                            ((q, k), dict(seq_lens=lens[:1]), "seq_lens"), ((q, k), dict(positions=pos[:, :2]), "positions"),
                            ((q, k), dict(seq_lens=lens, q_out=k), "q_out"), ((q, None), dict(seq_lens=lens, k_out=k), "without"),
                            ((q.double(), k.double()), dict(seq_lens=lens), "f32, bf16"),
                            ((q, k), dict(seq_lens=lens, status=pos.long()), "status"), ((q, k), dict(seq_lens=lens), "CUDA")):
        with pytest.raises(ValueError, match=msg):
            sv.spec_rope(*args, r, **over)
