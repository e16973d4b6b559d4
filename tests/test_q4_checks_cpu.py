"""Refusals of the 4-bit cache and the windowed attention: the library's host
checks (pointers are never dereferenced) and the binding's. No GPU."""
import ctypes

import pytest
import torch

import speculative_verify_paged_gb300 as sv


@pytest.fixture(scope="module")
def lib():
    sv.build()
    return sv.load_library()


FAKE, NULL = ctypes.c_void_p(0x1000), None
ODD = ctypes.c_void_p(0x1008)


def test_record_sizes(lib):
    assert lib.sv_q4_record_bytes(128, 16) == 16 * 68
    assert lib.sv_q4_record_bytes(64, 8) == 8 * 36
    for d, bs in ((0, 16), (48, 16), (288, 16), (128, 0), (128, 12), (128, 72), (-32, 16)):
        assert lib.sv_q4_record_bytes(d, bs) == 0
    with pytest.raises(ValueError, match="multiple of 32"):
        sv.q4_record_bytes(100)


def append(lib, k=FAKE, pool=FAKE, dt=1, layout=None, B=2, n=5, H=2, d=128, bs=16, nb=10):
    return lib.kv_block_append_q4(k, FAKE, dt, pool, FAKE, layout, FAKE, 4, FAKE, B, n, H, d, bs, nb, NULL, NULL)


def lay(*x):
    return ctypes.byref(sv._Layout(*x))


def test_append_refusals(lib):
    assert append(lib, k=NULL) == 1 and b"null" in lib.sv_last_error_string()
    assert append(lib, n=0) == 1 and append(lib, B=-1) == 1 and append(lib, nb=0) == 1
    assert append(lib, dt=2) == 2 and append(lib, dt=3) == 2
    assert append(lib, d=48) == 2 and append(lib, d=288) == 2 and append(lib, bs=12) == 2 and append(lib, bs=72) == 2
    assert append(lib, B=70000) == 2
    assert append(lib, pool=ODD) == 1 and b"aligned" in lib.sv_last_error_string()
    assert append(lib, layout=lay(2176, 1088, 1)) == 1      # a slot stride
    assert append(lib, layout=lay(2176, 1072, 0)) == 1      # records overlap
    assert append(lib, layout=lay(2180, 1088, 0)) == 1      # not a multiple of 16
    assert append(lib, B=0) == 0


def gather(lib, pool=FAKE, start=FAKE, dt=1, B=2, rows=5, d=128, bs=16):
    return lib.kv_block_gather_q4(pool, FAKE, None, FAKE, 4, FAKE, start, B, rows, 2, d, bs, 10, FAKE, FAKE, dt, NULL,
                                  NULL)


def test_gather_refusals(lib):
    assert gather(lib, pool=NULL) == 1 and gather(lib, start=NULL) == 1
    assert gather(lib, rows=-1) == 1
    assert gather(lib, dt=2) == 2 and gather(lib, d=40) == 2 and gather(lib, bs=4) == 2
    assert gather(lib, pool=ODD) == 1
    assert gather(lib, rows=0) == 0 and gather(lib, B=0) == 0


def attn_q4(lib, q=FAKE, qdt=1, odt=1, pool=FAKE, layout=None, B=2, n=5, Hq=8, H=2, d=128, bs=16, scale=0.1, W=0, S=0,
            ws=1 << 30, wsp=FAKE, mb=4):
    return lib.spec_verify_attn_q4(q, qdt, pool, FAKE, layout, FAKE, mb, FAKE, B, n, Hq, H, d, bs, 10, scale, W, S, FAKE,
                                   odt, wsp, ws, NULL, NULL)


def test_attention_refusals(lib):
    assert attn_q4(lib, q=NULL) == 1
    assert attn_q4(lib, Hq=7) == 1 and attn_q4(lib, n=0) == 1 and attn_q4(lib, mb=0) == 1
    assert attn_q4(lib, W=-1) == 1 and attn_q4(lib, W=4, S=-1) == 1
    assert attn_q4(lib, scale=0.0) == 1 and attn_q4(lib, scale=float("inf")) == 1 and attn_q4(lib, scale=float("nan")) == 1
    assert attn_q4(lib, qdt=2, odt=2) == 2 and attn_q4(lib, qdt=1, odt=0) == 2
    assert attn_q4(lib, d=48) == 2 and attn_q4(lib, bs=12) == 2
    assert attn_q4(lib, ws=16) == 3 and attn_q4(lib, wsp=NULL) == 3
    assert attn_q4(lib, wsp=ctypes.c_void_p(0x1010)) == 3
    assert attn_q4(lib, pool=ODD) == 1
    assert attn_q4(lib, layout=lay(2176, 1088, 128)) == 1
    assert attn_q4(lib, B=0) == 0


def attn_window(lib, kdt=1, W=4, S=0, scale=FAKE, ws=1 << 30):
    return lib.spec_verify_attn_window(FAKE, 1, FAKE, FAKE, kdt, None, scale, scale, FAKE, 4, FAKE, 2, 5, 8, 2, 128, 16,
                                       10, 0.1, W, S, FAKE, 1, FAKE, ws, NULL, NULL)


def test_window_refusals(lib):
    assert attn_window(lib, W=-1) == 1 and attn_window(lib, S=-1) == 1
    assert attn_window(lib, kdt=2) == 2 and attn_window(lib, kdt=4) == 2   # f16; not a public type
    assert attn_window(lib, kdt=3, scale=NULL) == 1
    assert attn_window(lib, ws=16) == 3


def test_workspace_sizes(lib):
    full = lib.spec_verify_attn_workspace_size(64, 5, 64, 8, 128, 512, 16)
    # no window, or one that reaches every key: the usual workspace
    assert lib.spec_verify_attn_window_workspace_size(64, 5, 64, 8, 128, 512, 16, 0, 0) == full
    assert lib.spec_verify_attn_window_workspace_size(64, 5, 64, 8, 128, 512, 16, 512 * 16, 4) == full
    assert lib.spec_verify_attn_window_workspace_size(64, 5, 64, 8, 128, 512, 16, 2 ** 31 - 1, 2 ** 31 - 1) == full
    assert 0 < lib.spec_verify_attn_window_workspace_size(1, 5, 64, 8, 128, 8192, 16, 1024, 4) <= \
        lib.spec_verify_attn_workspace_size(1, 5, 64, 8, 128, 8192, 16)
    for bad in ((-1, 5, 8, 2, 128, 4, 16, 0, 0), (1, 5, 7, 2, 128, 4, 16, 0, 0), (1, 5, 8, 2, 128, 4, 16, -1, 0),
                (1, 5, 8, 2, 128, 4, 16, 1, -1), (1, 5, 8, 2, 128, 4, 0, 1, 1)):
        assert lib.spec_verify_attn_window_workspace_size(*bad) == 0
        assert lib.spec_verify_attn_q4_workspace_size(*bad) == 0


def test_capacity_limit(lib):
    # positions are 32-bit: 2^30 tokens of table a sequence and more are refused, whatever the lengths
    big = 1 << 26
    assert attn_q4(lib, mb=big) == 2 and b"2^30" in lib.sv_last_error_string()
    assert attn_q4(lib, mb=2 ** 31 - 1, qdt=0, odt=0) == 2
    assert lib.kv_block_append_q4(FAKE, FAKE, 1, FAKE, FAKE, None, FAKE, big, FAKE, 2, 5, 2, 128, 16, 10, NULL, NULL) == 2
    assert lib.kv_block_gather_q4(FAKE, FAKE, None, FAKE, big, FAKE, FAKE, 2, 5, 2, 128, 16, 10, FAKE, FAKE, 1, NULL,
                                  NULL) == 2
    assert lib.spec_verify_attn_window(FAKE, 1, FAKE, FAKE, 1, None, NULL, NULL, FAKE, big, FAKE, 2, 5, 8, 2, 128, 16, 10,
                                       0.1, 4, 0, FAKE, 1, FAKE, 1 << 40, NULL, NULL) == 2
    assert b"2^30" in lib.sv_last_error_string()


# ---------------------------------------------------------------- binding ---

REC = 16 * 68


def _args(**over):
    a = dict(q=torch.zeros(2, 3, 8, 128, dtype=torch.bfloat16), k=torch.zeros(10, 2, REC, dtype=torch.uint8),
             v=torch.zeros(10, 2, REC, dtype=torch.uint8), bt=torch.zeros(2, 4, dtype=torch.int32),
             lens=torch.full((2,), 20, dtype=torch.int32), new=torch.zeros(2, 3, 2, 128, dtype=torch.bfloat16),
             start=torch.zeros(2, dtype=torch.int32), status=None)
    a.update(over)
    return a


@pytest.mark.parametrize("over,msg", [
    (dict(k=torch.zeros(10, 2, REC + 16, dtype=torch.uint8)), "4-bit pools must be"),
    (dict(v=torch.zeros(9, 2, REC, dtype=torch.uint8)), "4-bit pools must be"),
    (dict(k=torch.zeros(10, 2, 16, 68, dtype=torch.uint8)), "4-bit pools must be"),
    (dict(k=torch.zeros(10, 2, REC, dtype=torch.int8)), "uint8"),
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
        sv.spec_verify_attn_q4(a["q"], a["k"], a["v"], a["bt"], a["lens"], status=a["status"])
    with pytest.raises(ValueError, match=msg):
        sv.kv_block_append_q4(a["new"], a["new"], a["k"], a["v"], a["bt"], a["lens"], status=a["status"])
    with pytest.raises(ValueError, match=msg):
        sv.kv_block_gather_q4(a["k"], a["v"], a["bt"], a["lens"], a["start"], 4, 128, status=a["status"])


def test_binding_refusals_of_one_entry_point_each():
    a = _args()
    with pytest.raises(ValueError, match="kv heads"):
        sv.kv_block_append_q4(a["new"][:, :, :1], a["new"][:, :, :1], a["k"], a["v"], a["bt"], a["lens"])
    with pytest.raises(ValueError, match="one dtype"):
        sv.kv_block_append_q4(a["new"], a["new"].float(), a["k"], a["v"], a["bt"], a["lens"])
    with pytest.raises(ValueError, match="must be"):
        sv.kv_block_gather_q4(a["k"], a["v"], a["bt"], a["lens"], a["start"][:1], 4, 128)
    with pytest.raises(ValueError, match="k_out must be"):
        sv.kv_block_gather_q4(a["k"], a["v"], a["bt"], a["lens"], a["start"], 4, 128, k_out=torch.zeros(2, 4, 2, 64))
    with pytest.raises(ValueError, match="n_rows"):
        sv.kv_block_gather_q4(a["k"], a["v"], a["bt"], a["lens"], a["start"], -1, 128)
    with pytest.raises(ValueError, match="out must be"):
        sv.spec_verify_attn_q4(a["q"], a["k"], a["v"], a["bt"], a["lens"], out=torch.zeros(2, 3, 8, 128))
    with pytest.raises(ValueError, match="layout reaches"):
        sv.spec_verify_attn_q4(a["q"], a["k"], a["v"], a["bt"], a["lens"], layout=(2 * REC + 16, REC, 0), num_blocks=10,
                               H_kv=2)
    pool = torch.zeros(10, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="pools must be"):
        sv.spec_verify_attn_window(a["q"], pool[..., :64], pool[..., :64], a["bt"], a["lens"], 4)
    with pytest.raises(ValueError, match="one dtype"):
        sv.spec_verify_attn_window(a["q"], pool, pool.float(), a["bt"], a["lens"], 4)
    with pytest.raises(ValueError, match="k_scale"):
        sv.spec_verify_attn_window(a["q"], pool.to(torch.uint8), pool.to(torch.uint8), a["bt"], a["lens"], 4)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_verify_attn_window(a["q"], pool, pool, a["bt"], a["lens"], 4)
