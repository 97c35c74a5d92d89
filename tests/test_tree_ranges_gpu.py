"""Attention over the paged cache at the ends of the values' range: queries and keys whose sizes cancel,
values near the least normal number.  Scaled by powers of two, exactly, against tests/cache_ref.py."""
import numpy as np
import pytest
import torch

from cache_ref import Batch, hold

pytestmark = pytest.mark.gpu

SHAPES = [(2, 3), (4, 4), (8, 20)]  # heads a group, drafted tokens: 6 and 16 rows, then tiles of 128


def _pkg():
    import online_softmax_flashattention_attention_gb300 as pkg
    return pkg


def _run(batch):
    args, kw = batch.dev()
    O = torch.full_like(args[0], float("nan"))
    LSE = torch.full((args[0].shape[1], args[0].shape[0]), float("nan"), device="cuda")
    out = _pkg().attn_fwd_tree(*args, O, LSE, **kw)
    _pkg().cache_check()
    return out


def _scaled(b, name, power):
    """k or v times 2^power; what nobody owns stays NaN."""
    if b.f8:
        s = getattr(b, name + "s")
        live = s != 255
        s[live] = (s[live].int() + power).to(torch.uint8)
    else:
        setattr(b, name, (getattr(b, name).double() * 2.0 ** power).to(torch.bfloat16))


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T", SHAPES)
@pytest.mark.parametrize("power", [100, -100])
def test_queries_and_keys_far_apart(power, G, T, d, f8):
    b = Batch(81, 2, G, d, 16, f8, [150, 3], [T, 2])
    _scaled(b, "k", power)
    b.Q = (b.Q.double() * 2.0 ** -power).to(torch.bfloat16)
    hold(*_run(b), b.reference())


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T", SHAPES)
def test_tiny_values(G, T, d, f8):
    """Values around 2^-116.  Beyond the usual bounds: with up to 16 rows a weight times an e4m3 key's scale
    is a bf16, off by half its least step, 2^-134, times a code of 448 at most, where it is under 2^-126."""
    b = Batch(82, 2, G, d, 16, f8, [150, 3], [T, 2])
    _scaled(b, "v", -116)
    O, LSE = _run(b)
    O_ref, LSE_ref, tolO, tolL = b.reference()
    tolO = tolO - 1e-30 + (160 if f8 else 0) * 448 * 2.0 ** -134 + 2.0 ** -133
    err = np.abs(O.double().cpu().numpy() - O_ref)
    assert np.all(err <= tolO), f"{np.max(err / tolO):.3g} of the bound"
    assert np.all(np.abs(LSE.double().cpu().numpy() - LSE_ref) <= tolL)
