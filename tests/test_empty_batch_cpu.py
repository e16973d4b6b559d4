"""Calls of no sequences over quantised pools: nothing to do, nothing needed, whatever the shape. No GPU."""
import ctypes

import pytest

import speculative_verify_paged_gb300 as sv


@pytest.mark.parametrize("q_dtype", [0, 1])
@pytest.mark.parametrize("n,Hq,Hkv,d,bs", [(5, 64, 8, 128, 16), (1, 32, 8, 128, 16), (3, 8, 2, 64, 16)])
@pytest.mark.parametrize("name", ["spec_verify_attn_q4", "spec_verify_attn_q8"])
def test_an_empty_batch_asks_for_no_workspace(name, n, Hq, Hkv, d, bs, q_dtype):
    sv.build()
    lib = sv.load_library()
    fake = ctypes.c_void_p(0x10000)
    size = getattr(lib, name + "_workspace_size")(0, n, Hq, Hkv, d, 512, bs, 0, 0)
    assert size == 0
    # (the binding's smallest workspace is 256 bytes)
    assert getattr(lib, name)(fake, q_dtype, fake, fake, None, fake, 512, fake, 0, n, Hq, Hkv, d, bs, 10, 0.1, 0, 0, fake, q_dtype,
                              fake, 256, None, None) == 0
