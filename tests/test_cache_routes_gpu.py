"""Routes through the paged cache that a program takes and the other files leave out."""
import numpy as np
import pytest
import torch

from cache_ref import HALF_BF16, Batch

pytestmark = pytest.mark.gpu


def _pkg():
    import online_softmax_flashattention_attention_gb300 as pkg
    return pkg


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("hkv,G,d", [(2, 4, 128), (1, 8, 64), (3, 1, 64)])
def test_a_prompt_over_a_prefix_read_back_with_grouped_heads(hkv, G, d, f8):
    """What attn_cache_read returns, each K/V head repeated for its group, through the packed forward:
    a chain's tokens as attn_fwd_tree has them.  As they are, with fewer heads, they are refused."""
    pkg = _pkg()
    b = Batch(61, hkv, G, d, 32, f8, [150, 7], [9, 4], masks="chain")
    args, kw = b.dev()
    O, LSE = pkg.attn_fwd_tree(*args, **kw)
    cu_k = _i32([0, 159, 170])
    sc = {n: kw[n] for n in ("k_scale", "v_scale") if n in kw}
    K, V = pkg.attn_cache_read(args[1], args[2], args[3], cu_k, 170, **sc)
    cu_q = args[5]
    if G > 1:
        with pytest.raises(ValueError, match="repeat"):
            pkg.attn_fwd_varlen(args[0], K, V, cu_q, cu_k, 9, causal=True)
    K, V = (x.repeat_interleave(G, 1) for x in (K, V))
    O2, LSE2 = pkg.attn_fwd_varlen(args[0], K, V, cu_q, cu_k, 9, causal=True)
    pkg.cache_check()
    # each is off by half a bf16 step of O, and by one of every probability: 2^-8 (|O| + A), both at most max |v|
    assert bool(((O - O2).float().abs() <= 4 * HALF_BF16 * V.float().abs().max()).all())
    # scores: d 2^-24 |q| |k| / sqrt(d) each, |q| |k| under 250 here, and 2^-17 of the query row's largest where
    # a value is 2^-9 of it and less
    assert bool(((LSE - LSE2).abs() <= 4e-4).all())
