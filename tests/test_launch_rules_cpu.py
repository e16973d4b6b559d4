"""The rule of the programmatic launches, checked in the sources: a kernel may
start while the one before it in the stream still runs, so what that one may
have written is read after the wait on it, and with plain loads. No GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_verify_paged_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*", "", text)


def body(name, kernel):
    """The statements of a kernel, from its name to the closing brace of its function."""
    text = source(name)
    at = text.index("{", re.search(r"\b%s\s*\([^;]*?\)\s*\{" % kernel, text).end() - 1)
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i]
    raise AssertionError("unbalanced braces in %s" % name)


@pytest.mark.parametrize("name,kernel,rows", [
    ("kv_append.cu", "kv_append_kernel", r"load8_in<|\bkn\[|\bvn\["),
    ("q4_cache.cu", "q4_append_kernel", r"load8\("),
    ("mla.cu", "latent_append_kernel", r"__ldg\(c_new|\bc_new\["),
])
def test_appends_read_the_new_rows_after_the_wait(name, kernel, rows):
    # (kv_block_gather_q4 lets the next kernel start and then writes the rows that an append may take)
    b = body(name, kernel)
    reads = [m.start() for m in re.finditer(rows, b)]
    assert reads
    # the last wait of the kernel: those before it stand in branches that return
    assert b.rindex("pdl_wait()") < min(reads)


@pytest.mark.parametrize("name,helper", [("kv_append.cu", "load8_in"), ("q4_cache.cu", "load8")])
def test_appends_read_the_new_rows_with_plain_loads(name, helper):
    assert "__ldg" not in body(name, helper)
    assert "__ldg" not in body("mla.cu", "latent_append_kernel")


@pytest.mark.parametrize("name,kernel,stores", [
    ("attn.cu", "attn_order_kernel", r"(?<!auto )\bplace\("),
    ("mla.cu", "mla_order_kernel", r"\border\["),
])
def test_orders_are_written_after_the_wait(name, kernel, stores):
    # (the workspace may be shared with a call of another layout that still reads it)
    b = body(name, kernel)
    at = [m.start() for m in re.finditer(stores, b)]
    assert at and b.index("pdl_wait()") < min(at)
