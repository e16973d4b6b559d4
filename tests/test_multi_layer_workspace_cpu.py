"""The workspace that the layers of a MultiLayerVerify share holds what the largest of them needs. No GPU."""
import pytest
import torch

import speculative_verify_paged_gb300 as sv
from test_multi_layer_rope_cpu import layer, round_of


@pytest.mark.parametrize("order", [(0, 1, 2), (2, 1, 0), (1, 2, 0)])
def test_layers_larger_than_the_first(order):
    sv.build()
    layers = [[layer(8, 2, torch.bfloat16), layer(64, 8, torch.bfloat16), layer(96, 4, torch.float32, window=30)][i] for i in order]
    need = [sv.attn_q8_workspace_size(2, 3, 8, 2, 128, 4), sv.attn_q8_workspace_size(2, 3, 64, 8, 128, 4),
            sv.attn_window_workspace_size(2, 3, 96, 4, 128, 4, 16, 30)]
    assert round_of(layers).attn_ws.numel() == max(max(need), 256)
