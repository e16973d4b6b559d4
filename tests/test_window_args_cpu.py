"""window and sinks of any size reach the library as they are meant. No GPU."""
import pytest
import torch

import speculative_verify_paged_gb300 as sv

TOP = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def built():
    sv.build()


@pytest.mark.parametrize("window,sinks,got", [
    (4, 1, (4, 1)), (TOP, TOP, (TOP, TOP)), (2 ** 31, 0, (TOP, 0)), (2 ** 32, 3, (TOP, 3)), (2 ** 32 + 5, 0, (TOP, 0)),
    (5, 2 ** 32, (5, TOP)), (2 ** 63 - 1, 2 ** 40 + 1, (TOP, TOP)),
])
def test_values_past_32_bits(monkeypatch, window, sinks, got):
    seen = []

    class Lib:
        def __getattr__(self, name):
            if name == "sv_q4_record_bytes":
                return lambda d, bs: bs * (d // 2 + 4)
            return lambda *a: seen.append((name, a)) or (256 if name.endswith("size") else 0)

    sv.q4_record_bytes(128)
    for f in (sv.attn_window_workspace_size, sv.attn_q4_workspace_size):
        f.cache_clear()
    monkeypatch.setattr(sv, "load_library", lambda *a: Lib())
    monkeypatch.setattr(sv, "_ready", lambda *a: None)
    monkeypatch.setattr(sv, "_stream", lambda: None)
    q = torch.zeros(2, 3, 8, 128, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.full((2,), 20, dtype=torch.int32)
    pool, pool4 = torch.zeros(10, 2, 16, 128, dtype=torch.bfloat16), torch.zeros(10, 2, 1088, dtype=torch.uint8)
    sv.spec_verify_attn_window(q, pool, pool, table, lens, window, sinks)
    sv.spec_verify_attn_q4(q, pool4, pool4, table, lens, window=window, sinks=sinks)
    for f in (sv.attn_window_workspace_size, sv.attn_q4_workspace_size):
        f.cache_clear()
    sizes = [a[-2:] for name, a in seen if name.endswith("size")]
    calls = {name: a for name, a in seen if not name.endswith("size")}
    assert sizes == [got, got]
    assert calls["spec_verify_attn_window"][19:21] == got
    assert calls["spec_verify_attn_q4"][16:18] == got


def test_workspace_of_a_window_past_32_bits():
    shape = (64, 5, 64, 8, 128, 512, 16)
    assert sv.attn_window_workspace_size(*shape, 2 ** 32 + 5, 0) == sv.attn_workspace_size(*shape)
    assert sv.attn_q4_workspace_size(*shape, 2 ** 32 + 5, 0) == sv.attn_q4_workspace_size(*shape)
    assert sv.attn_window_workspace_size(*shape, -1, 0) == sv.attn_window_workspace_size(*shape, 2, -2 ** 32 - 1) == 0


def test_layouts_past_the_pool():
    # one layer of [blocks][slots][layers][H_kv][d]: the last rows of the last block are the pool's last elements
    nb, bs, layers, H, d = 6, 16, 3, 2, 128
    big = torch.zeros(nb, bs, layers, H, d, dtype=torch.bfloat16)
    q = torch.zeros(2, 3, 8, d, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.full((2,), 20, dtype=torch.int32)
    layout = (bs * layers * H * d, d, layers * H * d)

    def call(layer, blocks, lay=layout, first=None):
        v = big.view(-1)[layer * H * d:]
        sv.spec_verify_attn_window(q, v if first is None else v[:first], v, table, lens, 4, layout=lay, num_blocks=blocks,
                                   H_kv=H)

    for layer in range(layers):   # within the pool: as far as the check for CUDA tensors
        with pytest.raises(ValueError, match="CUDA"):
            call(layer, nb)
    with pytest.raises(ValueError, match="CUDA"):
        call(0, nb, first=H * d)   # a view of the first rows only
    with pytest.raises(ValueError, match="layout reaches"):
        call(0, nb + 1)
    with pytest.raises(ValueError, match="layout reaches"):
        call(2, nb, (bs * layers * H * d, d, layers * H * d + 128))
