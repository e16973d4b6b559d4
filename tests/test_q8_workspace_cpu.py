"""The workspace that verify attention over 8-bit block-scaled pools asks for: what the path that
will run needs, and no more than that where only the tensor cores can run. No GPU."""
import ctypes
import re

import pytest

import speculative_verify_paged_gb300 as sv


@pytest.fixture(scope="module", autouse=True)
def lib():
    sv.build()
    return sv.load_library()


def call(lib, B, n, Hq, Hkv, mb, q_dtype, window=0, sinks=0, d=128, bs=16):
    """(status, bytes that the call says it needs) without a workspace; the pointers are never read."""
    fake = ctypes.c_void_p(0x1000)
    rc = lib.spec_verify_attn_q8(fake, q_dtype, fake, fake, None, fake, mb, fake, B, n, Hq, Hkv, d, bs, 10, 0.1, window, sinks,
                                 fake, q_dtype, None, 0, None, None)
    m = re.search(rb"needs (\d+) bytes", lib.sv_last_error_string())
    return rc, int(m.group(1)) if rc == 3 and m else None


def size(lib, B, n, Hq, Hkv, mb, window=0, sinks=0, d=128, bs=16):
    return lib.spec_verify_attn_q8_workspace_size(B, n, Hq, Hkv, d, mb, bs, window, sinks)


CHUNKS = [(1, 2047, 64, 8, 8192), (1, 512, 64, 8, 8192), (8, 2048, 64, 8, 512), (1, 148, 8, 8, 8192), (2, 1 << 14, 1, 1, 2048),
          (4, 200, 16, 2, 100), (16, 2047, 64, 8, 300)]


@pytest.mark.parametrize("window,sinks", [(0, 0), (512, 4)])
@pytest.mark.parametrize("shape", CHUNKS)
def test_many_query_rows_ask_for_what_the_tensor_cores_need(lib, shape, window, sinks):
    B, n, Hq, Hkv, mb = shape
    rc, need = call(lib, *shape, 1, window, sinks)
    got = size(lib, *shape, window, sinks)
    assert rc == 3 and got == need
    # a row's query (2 x 128 bytes and two floats, up to 64 rows padded to at most 80 columns), and partials of at most two
    # sequences a CTA, which are one an SM (at most 152) or one a kv head and 64 rows
    R = n * (Hq // Hkv)
    groups = -(-R // 64)
    ctas = max(152, Hkv * groups)
    assert got <= B * Hkv * groups * 80 * (256 + 16) + 2 * ctas * 64 * (128 + 2) * 4 + (1 << 16)


@pytest.mark.parametrize("shape", CHUNKS)
def test_rows_that_only_the_tensor_cores_take_are_refused_in_f32(lib, shape):
    # (as unsupported, not for a workspace that no size would satisfy)
    rc, _ = call(lib, *shape, 0)
    assert rc == 2 and b"too large" in lib.sv_last_error_string()


@pytest.mark.parametrize("d,bs", [(64, 16), (128, 32), (256, 16)])
def test_sizes_that_no_kernel_takes_ask_for_nothing(lib, d, bs):
    assert size(lib, 1, 1000, 8, 2, 1000, d=d, bs=bs) == 0
    for q_dtype in (0, 1):
        assert call(lib, 1, 1000, 8, 2, 1000, q_dtype, d=d, bs=bs)[0] == 2


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5)])
@pytest.mark.parametrize("B,n,Hq,Hkv,mb,d,bs", [
    (1, 1, 32, 8, 63, 128, 16), (64, 5, 64, 8, 512, 128, 16), (1, 8, 64, 8, 8192, 128, 16), (3, 147, 4, 4, 40, 128, 16),
    (2, 3, 8, 2, 30, 64, 16), (1, 9, 16, 2, 1000, 96, 32), (5, 2, 8, 8, 70, 256, 8)])
def test_the_size_serves_either_type_of_query(lib, B, n, Hq, Hkv, mb, d, bs, window, sinks):
    got = size(lib, B, n, Hq, Hkv, mb, window, sinks, d, bs)
    for q_dtype in (0, 1):
        rc, need = call(lib, B, n, Hq, Hkv, mb, q_dtype, window, sinks, d, bs)
        assert rc == 3 and got >= need > 0
