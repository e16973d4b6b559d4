"""Refusals of the 8-bit block-scaled cache: the library's host checks
(pointers are never dereferenced) and the binding's. No GPU."""
import ctypes

import pytest
import torch

import speculative_verify_paged_gb300 as sv
from oracle import q8 as oq8


@pytest.fixture(scope="module", autouse=True)
def lib():
    sv.build()
    return sv.load_library()


FAKE, NULL = ctypes.c_void_p(0x1000), None
ODD = ctypes.c_void_p(0x1008)
PAGE = 2 * 2048 + 128


def test_page_sizes(lib):
    for H, d, bs in ((8, 128, 16), (1, 128, 16), (32, 128, 16), (33, 64, 8), (5, 256, 64), (3, 16, 1), (2, 48, 12)):
        assert lib.sv_q8_page_bytes(H, d, bs) == oq8.page_bytes(H, d, bs) == sv.q8_page_bytes(H, d, bs)
    for H, d, bs in ((0, 128, 16), (2, 0, 16), (2, 40, 16), (2, 272, 16), (2, 128, 0), (2, 128, 65), (2, -16, 16), (65536, 128, 16)):
        assert lib.sv_q8_page_bytes(H, d, bs) == 0
    with pytest.raises(ValueError, match="multiple of 16"):
        sv.q8_page_bytes(2, 100)


@pytest.mark.parametrize("H,d,bs", [(1, 16, 16), (1, 128, 16), (8, 128, 16), (2, 64, 8), (3, 256, 64), (7, 48, 5), (65535, 128, 16)])
def test_heads_of_a_pool(H, d, bs):
    page = sv.q8_page_bytes(H, d, bs)
    if H < 100:
        pool = torch.zeros(2, page, dtype=torch.uint8)
        codes, scales = sv.q8_views(pool, H, d, bs)
        assert codes.shape == (2, H, bs, d) and codes.dtype == torch.float8_e4m3fn and scales.shape == (2, H)
        scales[1, H - 1] = 3.0
        codes.view(torch.uint8)[1, H - 1, bs - 1, d - 1] = 77
        assert pool[1, H * bs * d - 1] == 77 and float(oq8.split(pool.numpy(), H, d, bs)[1][1, H - 1]) == 3.0
    assert sv._q8_heads("", torch.empty(1, page, dtype=torch.uint8, device="meta"), d, bs, None) == H


def test_heads_of_a_pool_of_small_pages():
    # a head narrower than the padding: the page does not tell how many there are
    pool, q = torch.zeros(2, 128, dtype=torch.uint8), torch.zeros(1, 1, 6, 16)
    bt, one = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="pass H_kv"):
        sv.kv_block_gather_q8(pool, pool, bt, one, one, 1, 16, block_size=1)
    with pytest.raises(ValueError, match="pass H_kv"):
        sv.spec_verify_attn_q8(q, pool, pool, bt, one, block_size=1)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_verify_attn_q8(q, pool, pool, bt, one, block_size=1, H_kv=3)


def append(lib, k=FAKE, pool=FAKE, dt=1, layout=None, B=2, n=5, H=2, d=128, bs=16, nb=10, mb=4):
    return lib.kv_block_append_q8(k, FAKE, dt, pool, FAKE, layout, FAKE, mb, FAKE, B, n, H, d, bs, nb, NULL, NULL)


def lay(*x):
    return ctypes.byref(sv._Layout(*x))


def test_append_refusals(lib):
    assert append(lib, k=NULL) == 1 and b"null" in lib.sv_last_error_string()
    assert append(lib, n=0) == 1 and append(lib, B=-1) == 1 and append(lib, nb=0) == 1 and append(lib, mb=0) == 1
    assert append(lib, dt=2) == 2 and append(lib, dt=3) == 2 and append(lib, dt=5) == 2
    assert append(lib, d=40) == 2 and append(lib, d=272) == 2 and append(lib, bs=65) == 2
    assert append(lib, B=70000) == 2 and append(lib, H=70000) == 2
    assert append(lib, mb=1 << 26) == 2 and b"2^30" in lib.sv_last_error_string()
    assert append(lib, pool=ODD) == 1 and b"aligned" in lib.sv_last_error_string()
    assert append(lib, layout=lay(PAGE, 0, 128)) == 1 and append(lib, layout=lay(PAGE, 2048, 0)) == 1
    assert append(lib, layout=lay(PAGE - 16, 0, 0)) == 1 and append(lib, layout=lay(PAGE + 8, 0, 0)) == 1
    assert append(lib, B=0) == 0


def gather(lib, pool=FAKE, start=FAKE, dt=1, B=2, rows=5, d=128, bs=16, layout=None, mb=4):
    return lib.kv_block_gather_q8(pool, FAKE, layout, FAKE, mb, FAKE, start, B, rows, 2, d, bs, 10, FAKE, FAKE, dt, NULL,
                                  NULL)


def test_gather_refusals(lib):
    assert gather(lib, pool=NULL) == 1 and gather(lib, start=NULL) == 1 and gather(lib, rows=-1) == 1
    assert gather(lib, dt=2) == 2 and gather(lib, d=40) == 2 and gather(lib, bs=70) == 2 and gather(lib, mb=1 << 26) == 2
    assert gather(lib, pool=ODD) == 1 and gather(lib, layout=lay(PAGE, 1, 0)) == 1
    assert gather(lib, rows=0) == 0 and gather(lib, B=0) == 0


def attn(lib, q=FAKE, qdt=1, odt=1, pool=FAKE, layout=None, B=2, n=5, Hq=8, H=2, d=128, bs=16, scale=0.1, W=0, S=0,
         ws=1 << 30, wsp=FAKE, mb=4):
    return lib.spec_verify_attn_q8(q, qdt, pool, FAKE, layout, FAKE, mb, FAKE, B, n, Hq, H, d, bs, 10, scale, W, S, FAKE,
                                   odt, wsp, ws, NULL, NULL)


@pytest.mark.parametrize("d,qdt", [(128, 1), (64, 1), (128, 0)])
def test_attention_refusals(lib, d, qdt):
    def call(**over):
        return attn(lib, **{**dict(d=d, qdt=qdt, odt=qdt), **over})
    assert call(q=NULL) == 1 and call(Hq=7) == 1 and call(n=0) == 1 and call(mb=0) == 1
    assert call(W=-1) == 1 and call(W=4, S=-1) == 1
    assert call(scale=0.0) == 1 and call(scale=float("inf")) == 1 and call(scale=float("nan")) == 1
    assert call(qdt=2, odt=2) == 2 and call(odt=1 - qdt) == 2
    assert call(d=40) == 2 and call(d=272) == 2 and call(bs=65) == 2 and call(mb=1 << 26) == 2
    assert call(ws=16) == 3 and call(wsp=NULL) == 3 and call(wsp=ctypes.c_void_p(0x1010)) == 3
    assert call(pool=ODD) == 1 and call(layout=lay(1 << 20, 128, 0)) == 1 and call(layout=lay(512, 0, 0)) == 1
    assert call(B=0) == 0


def test_workspace_size_refusals(lib):
    for bad in ((-1, 5, 8, 2, 128, 4, 16, 0, 0), (1, 5, 7, 2, 128, 4, 16, 0, 0), (1, 5, 8, 2, 128, 4, 16, -1, 0),
                (1, 5, 8, 2, 128, 4, 16, 1, -1), (1, 5, 8, 2, 128, 4, 0, 1, 1)):
        assert lib.spec_verify_attn_q8_workspace_size(*bad) == 0


def _args(**over):
    a = dict(q=torch.zeros(2, 3, 8, 128, dtype=torch.bfloat16), k=torch.zeros(10, PAGE, dtype=torch.uint8),
             v=torch.zeros(10, PAGE, dtype=torch.uint8), bt=torch.zeros(2, 4, dtype=torch.int32),
             lens=torch.full((2,), 20, dtype=torch.int32), new=torch.zeros(2, 3, 2, 128, dtype=torch.bfloat16),
             start=torch.zeros(2, dtype=torch.int32), status=None)
    a.update(over)
    return a


@pytest.mark.parametrize("over,msg", [
    (dict(k=torch.zeros(10, PAGE + 128, dtype=torch.uint8)), "8-bit block-scaled pools must be"),
    (dict(v=torch.zeros(9, PAGE, dtype=torch.uint8)), "8-bit block-scaled pools must be"),
    (dict(k=torch.zeros(10, 2, PAGE // 2, dtype=torch.uint8)), "8-bit block-scaled pools must be"),
    (dict(k=torch.zeros(10, PAGE, dtype=torch.int8)), "uint8"),
    (dict(bt=torch.zeros(2, 4, dtype=torch.int64)), "block_table must be int32"),
    (dict(bt=torch.zeros(3, 4, dtype=torch.int32)), "block_table must be"),
    (dict(lens=torch.zeros(2, dtype=torch.int64)), "seq_lens must be int32"),
    (dict(lens=torch.zeros(1, dtype=torch.int32)), "seq_lens must be"),
    (dict(status=torch.zeros(1, dtype=torch.int64)), "status"),
    ({}, "CUDA"),
])
def test_binding_refusals(over, msg):
    a = _args(**over)
    with pytest.raises(ValueError, match=msg):
        sv.spec_verify_attn_q8(a["q"], a["k"], a["v"], a["bt"], a["lens"], status=a["status"], H_kv=2)
    with pytest.raises(ValueError, match=msg):
        sv.kv_block_append_q8(a["new"], a["new"], a["k"], a["v"], a["bt"], a["lens"], status=a["status"])
    with pytest.raises(ValueError, match=msg):
        sv.kv_block_gather_q8(a["k"], a["v"], a["bt"], a["lens"], a["start"], 4, 128, status=a["status"], H_kv=2)


def test_binding_refusals_of_one_entry_point_each():
    a = _args()
    with pytest.raises(ValueError, match="H_kv 1"):
        sv.kv_block_append_q8(a["new"][:, :, :1], a["new"][:, :, :1], a["k"], a["v"], a["bt"], a["lens"])
    with pytest.raises(ValueError, match="one dtype"):
        sv.kv_block_append_q8(a["new"], a["new"].float(), a["k"], a["v"], a["bt"], a["lens"])
    with pytest.raises(ValueError, match="must be"):
        sv.kv_block_gather_q8(a["k"], a["v"], a["bt"], a["lens"], a["start"][:1], 4, 128)
    with pytest.raises(ValueError, match="k_out must be"):
        sv.kv_block_gather_q8(a["k"], a["v"], a["bt"], a["lens"], a["start"], 4, 128, k_out=torch.zeros(2, 4, 2, 64))
    with pytest.raises(ValueError, match="n_rows"):
        sv.kv_block_gather_q8(a["k"], a["v"], a["bt"], a["lens"], a["start"], -1, 128)
    with pytest.raises(ValueError, match="out must be"):
        sv.spec_verify_attn_q8(a["q"], a["k"], a["v"], a["bt"], a["lens"], out=torch.zeros(2, 3, 8, 128))
    with pytest.raises(ValueError, match="layout reaches"):
        sv.spec_verify_attn_q8(a["q"], a["k"], a["v"], a["bt"], a["lens"], layout=(PAGE + 16, 0, 0), num_blocks=10, H_kv=2)
    with pytest.raises(ValueError, match="explicit layout"):
        sv.spec_verify_attn_q8(a["q"], a["k"], a["v"], a["bt"], a["lens"], layout=(PAGE, 0, 0), num_blocks=10)
    with pytest.raises(ValueError, match="explicit layout"):
        sv.kv_block_gather_q8(a["k"], a["v"], a["bt"], a["lens"], a["start"], 4, 128, layout=(PAGE, 0, 0), H_kv=2)


def test_calls_over_whole_elements_refuse_block_scaled_pools():
    a = _args()
    scale = torch.ones(2)
    for which in (0, 1):
        k, v = [a["k"], torch.zeros(10, 2, 16, 128, dtype=torch.uint8)][::1 - 2 * which]
        with pytest.raises(ValueError, match="block-scaled"):
            sv.kv_block_append(a["new"], a["new"], k, v, a["bt"], a["lens"], scale, scale)
        with pytest.raises(ValueError, match="block-scaled"):
            sv.spec_verify_attn(a["q"], k, v, a["bt"], a["lens"], None, scale, scale)
        with pytest.raises(ValueError, match="block-scaled"):
            sv.kv_tree_commit(k, v, a["bt"], a["lens"], torch.zeros(2, 3, dtype=torch.int32), a["lens"])
        with pytest.raises(ValueError, match="block-scaled"):
            sv.tree_verify_step(a["q"], a["new"], a["new"], k, v, a["bt"], a["lens"], None, None, None, None, None)
    with pytest.raises(ValueError, match="pools must be"):
        sv.spec_verify_attn_window(a["q"], a["k"], a["v"], a["bt"], a["lens"], 4, k_scale=scale, v_scale=scale)
    with pytest.raises(ValueError, match="4-bit pools must be"):
        sv.spec_verify_attn_q4(a["q"], a["k"], a["v"], a["bt"], a["lens"])
    # flat pools of e4m3 codes are taken as before
    flat = torch.zeros(10, 2 * 2048, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        sv.kv_block_append(a["new"], a["new"], flat, flat, a["bt"], a["lens"], scale, scale)


def test_a_rope_over_a_tree_needs_positions():
    a = _args()
    pool = torch.zeros(10, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="positions"):
        sv.tree_verify_step(a["q"], a["new"], a["new"], pool, pool, a["bt"], a["lens"], None, None, None, None, None,
                            rope=sv.Rope(128))
