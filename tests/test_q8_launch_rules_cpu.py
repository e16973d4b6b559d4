"""The rule of the programmatic launches in the 8-bit cache's and the rotation's
sources: what the kernel before may have written is read after the wait on it,
with plain loads. No GPU."""
import ctypes
import re

import pytest

import speculative_verify_paged_gb300 as sv
from test_launch_rules_cpu import body, source


@pytest.mark.parametrize("name,kernel,reads", [
    ("q8_cache.cu", "q8_append_kernel", r"\bload16\(|\*scale_at\b|\*at = w|= \*at\b"),
    ("q8_cache.cu", "q8_gather_kernel", r"= codes\[|q8_scale\(|write16\("),
    ("rope.cu", "rope_kernel", r"load_v<|store_v<|a\.positions\[rowi\]"),
])
def test_rows_and_pools_are_touched_after_the_wait(name, kernel, reads):
    b = body(name, kernel)
    at = [m.start() for m in re.finditer(reads, b)]
    assert at and b.rindex("pdl_wait()") < min(at)


@pytest.mark.parametrize("name", ["q8_cache.cu", "rope.cu", "attn_q8.cu"])
def test_plain_loads(name):
    assert "__ldg" not in source(name) and "ld.global.nc" not in source(name)


@pytest.mark.parametrize("seq,row,head", [
    (640, 64, 127), (64, 640, 64), (640, 320, 63), (640, 319, 64), (639, 320, 64), (0, 320, 64), (640, 0, 64), (2 ** 62, 2 ** 62, 64),
    (2 ** 63 - 1, 320, 64), (-640, 320, 64),
])
def test_rope_refuses_outputs_that_overlap(seq, row, head):
    # 2 sequences of 2 rows of 5 heads of 64 elements; the pointers are never read
    sv.build()
    lib = sv.load_library()
    r = sv.Rope(64)
    rows = ctypes.byref(sv._RopeRows(seq, row, head))
    fake = ctypes.c_void_p(0x1000)
    assert lib.spec_rope(fake, fake, None, None, 1, None, rows, None, None, r._ref, None, fake, 2, 2, 5, 0, 64, None, None) != 0
    assert re.search(b"overlap|too large|negative", lib.sv_last_error_string())
