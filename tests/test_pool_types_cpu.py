"""Calls refuse pools that they cannot read. No GPU: pointers are never
dereferenced."""
import ctypes

import pytest
import torch

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


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("which", [0, 1])
def test_calls_over_whole_elements_refuse_4_bit_pools(d, which):
    # with scales given, as for e4m3 pools: taken for those, 4-bit pools would be read and written past their end
    B, n, H = 2, 3, 2
    rec = sv.q4_record_bytes(d, 16)
    pools = [torch.zeros(10, H, 16, d, dtype=torch.uint8) for _ in range(2)]
    pools[which] = torch.zeros(10, H, rec, dtype=torch.uint8)
    new, q = (torch.zeros(B, n, h, d, dtype=torch.bfloat16) for h in (H, 8))
    bt, lens, sc = torch.zeros(B, 4, dtype=torch.int32), torch.full((B,), 20, dtype=torch.int32), torch.ones(H)
    nodes, acc = torch.zeros(B, n, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    with pytest.raises(ValueError, match="kv_block_append does not take 4-bit pools"):
        sv.kv_block_append(new, new, *pools, bt, lens, sc, sc)
    with pytest.raises(ValueError, match="spec_verify_attn does not take 4-bit pools"):
        sv.spec_verify_attn(q, *pools, bt, lens, None, sc, sc)
    with pytest.raises(ValueError, match="spec_verify_attn does not take 4-bit pools"):
        sv.spec_verify_attn(q, *pools, bt, lens, None, sc, sc, tree_parent=nodes)
    with pytest.raises(ValueError, match="kv_tree_commit does not take 4-bit pools"):
        sv.kv_tree_commit(*pools, bt, lens, nodes, acc)
    with pytest.raises(ValueError, match="tree_verify_step does not take 4-bit pools"):
        sv.tree_verify_step(q, new, new, *pools, bt, lens, nodes, torch.zeros(B, n, 50), torch.zeros(B, n, 50), nodes,
                            torch.zeros(B, n, 2), sc, sc)
    # blocks of e4m3 codes in one dimension went through before and still do (to the check for CUDA tensors)
    flat = [torch.zeros(10, H, 16 * d, dtype=torch.uint8) for _ in range(2)]
    with pytest.raises(ValueError, match="CUDA"):
        sv.kv_block_append(new, new, *flat, bt, lens, sc, sc)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_verify_attn(q, *flat, bt, lens, None, sc, sc)
