"""Calls refuse pools that they cannot read. No GPU: pointers are never
dereferenced."""
import ctypes

import pytest

import speculative_verify_paged_gb300 as sv


@pytest.fixture(scope="module")
def lib():
    sv.build()
    return sv.load_library()


FAKE, NULL = ctypes.c_void_p(0x1000), None


@pytest.mark.parametrize("kv_dtype", [2, 4, 5, 99, -1])
@pytest.mark.parametrize("d", [128, 64])
def test_attention_refuses_other_element_types(lib, kv_dtype, d):
    # (4 is what the library calls a 4-bit pool inside: no entry point takes it)
    args = [FAKE, 1, FAKE, FAKE, kv_dtype, None, FAKE, FAKE, FAKE, 4, FAKE, 2, 5, 8, 2, d, 16, 10, 0.1, FAKE, 1, FAKE, 16,
            NULL]
    for rc in (lib.spec_verify_attn(*args, NULL), lib.spec_verify_attn_ex(*args, 4, NULL),
               lib.spec_verify_attn_tree(*args[:11], FAKE, *args[11:], NULL),
               lib.spec_verify_attn_window(*args[:19], 4, 0, *args[19:], NULL)):
        assert rc == 2 and b"kv_dtype %d" % kv_dtype in lib.sv_last_error_string()
    args[4] = 1   # the same call over bf16 pools gets as far as its workspace
    assert lib.spec_verify_attn(*args, NULL) == 3
