"""attn_fwd_varlen's binding refuses tensors that do not fit together before it calls the library:
it hands over one head count, so K and V with fewer heads would be read past their end."""
import pytest
import torch

import online_softmax_flashattention_attention_gb300 as pkg


def _z(*shape, dt=torch.bfloat16):
    return torch.zeros(shape, dtype=dt)


CU = torch.tensor([0, 5], dtype=torch.int32)


@pytest.mark.parametrize("k,v", [((5, 2, 64), (5, 2, 64)),      # grouped heads, as attn_cache_read returns them
                                 ((5, 1, 64), (5, 1, 64)), ((5, 16, 64), (5, 16, 64)), ((5, 8, 128), (5, 8, 128)),
                                 ((5, 8, 64), (5, 2, 64)), ((5, 8, 64), (4, 8, 64))])
def test_heads_and_widths_that_are_not_the_querys(k, v):
    with pytest.raises(ValueError, match="repeat"):
        pkg.attn_fwd_varlen(_z(5, 8, 64), _z(*k), _z(*v), CU, CU, 5)


@pytest.mark.parametrize("t", ["Q", "K", "V"])
def test_types_and_placement(t):
    x = {n: _z(5, 8, 64) for n in "QKV"}
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkg.attn_fwd_varlen(x["Q"], x["K"], x["V"], CU, CU, 5)
    x[t] = x[t].half()
    with pytest.raises(ValueError):
        pkg.attn_fwd_varlen(x["Q"], x["K"], x["V"], CU, CU, 5)
