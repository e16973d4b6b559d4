"""What MultiLayerVerify sets up for layers that rotate their rows: a pair of buffers for each shape
and type among them, and a refusal at its construction where a round could not run. No GPU."""
import pytest
import torch

import speculative_verify_paged_gb300 as sv

B, N, D = 2, 3, 128


@pytest.fixture(scope="module", autouse=True)
def lib():
    sv.build()


def layer(H_q, H_kv, dtype, rope=None, d=D, **over):
    l = dict(q=torch.zeros(B, N, H_q, d, dtype=dtype), k_new=torch.zeros(B, N, H_kv, d, dtype=dtype),
             v_new=torch.zeros(B, N, H_kv, d, dtype=dtype))
    if dtype == torch.float32:
        l["k_cache"], l["v_cache"] = (torch.zeros(10, H_kv, 16, d) for _ in range(2))
    else:
        l["k_cache"], l["v_cache"] = sv.alloc_q8_pools(10, H_kv, d, device="cpu")
    l["rope"] = rope
    l.update(over)
    return l


def round_of(layers):
    return sv.MultiLayerVerify(layers, torch.zeros(B, 4, dtype=torch.int32), torch.full((B,), 20, dtype=torch.int32),
                               torch.zeros(B, N, 50), torch.zeros(B, N - 1, 50), torch.zeros(B, N - 1, dtype=torch.int32),
                               torch.zeros(B, N, 2))


def test_a_pair_of_buffers_for_each_shape_and_type():
    r = sv.Rope(D)
    layers = [layer(8, 2, torch.float32), layer(8, 2, torch.bfloat16, r), layer(8, 2, torch.float32, r), layer(4, 1, torch.bfloat16, r),
              layer(8, 2, torch.bfloat16), layer(8, 2, torch.bfloat16, r)]
    m = round_of(layers)
    assert [t is None for t in m.turned] == [True, False, False, False, True, False]
    for l, t in zip(layers, m.turned):
        if t is not None:
            assert all(x.shape == y.shape and x.dtype == y.dtype and x.is_contiguous() for x, y in zip(t, (l["q"], l["k_new"])))
    assert m.turned[1] is m.turned[5] and m.turned[2] is not m.turned[1]


def test_buffers_and_outputs_are_packed_where_the_rows_are_not():
    l = layer(8, 2, torch.bfloat16, sv.Rope(D))
    l["q"] = torch.zeros(B, 8, N, D, dtype=torch.bfloat16).transpose(1, 2)
    l["k_new"] = torch.zeros(B, N, 12, D, dtype=torch.bfloat16)[:, :, 8:10]
    m = round_of([l])
    assert all(t.is_contiguous() for t in m.turned[0]) and m.outs[0].is_contiguous()


@pytest.mark.parametrize("over", [
    dict(k_new=torch.zeros(B, N, 2, D)), dict(k_new=torch.zeros(B, N + 1, 2, D, dtype=torch.bfloat16)),
    dict(k_new=torch.zeros(B, N, 2, 64, dtype=torch.bfloat16)), dict(q=torch.zeros(B + 1, N, 8, D, dtype=torch.bfloat16)),
    dict(rope=sv.Rope(64, offset=65))])
def test_a_layer_that_cannot_be_rotated_is_refused_at_once(over):
    with pytest.raises(ValueError, match="layer 1 rotates"):
        round_of([layer(8, 2, torch.bfloat16), layer(8, 2, torch.bfloat16, over.pop("rope", None) or sv.Rope(D), **over)])
    with pytest.raises(TypeError, match="layer 0"):
        round_of([layer(8, 2, torch.bfloat16, rope={"rotary_dim": 128})])
