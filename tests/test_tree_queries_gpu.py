"""Attention over the paged cache for queries and scales at the edge: scales so small that a row's
factor leaves fp32, rows of zeros, infinities and NaN in the query.  Against tests/cache_ref.py."""
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


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T", SHAPES)
@pytest.mark.parametrize("scale", [1e-8, 1e-30, 1e-44])
def test_tiny_scales_and_zero_rows(scale, G, T, d, f8):
    """The scores all but vanish: every row is the mean of what it sees."""
    b = Batch(71, 2, G, d, 16, f8, [150, 0, 31], [T, T, 1], scale=scale)
    b.Q[::2] = 0
    b.Q[1::4] *= 2.0 ** -120
    hold(*_run(b), b.reference())


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T", SHAPES)
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
def test_queries_that_are_not_finite(poison, G, T, d, f8):
    """A row that sees nothing is O = 0, LSE = -inf whatever its query holds; one that sees keys of
    either sign is NaN; the other rows do not notice."""
    b = Batch(72, 2, G, d, 32, f8, [0, 150], [T, T])
    blind, seeing = 1, T + 2  # packed rows: the second token of the first sequence, the third of the other
    b.masks[blind] = 0
    clean = [x.clone() for x in _run(b)]
    assert bool((clean[0][blind] == 0).all()) and bool(torch.isneginf(clean[1][:, blind]).all())
    b.Q[blind, :, d // 2] = poison
    b.Q[blind, :, 0] = 0
    b.Q[seeing, :, 3] = poison
    O, LSE = _run(b)
    assert bool((O[blind] == 0).all()) and bool(torch.isneginf(LSE[:, blind]).all())
    assert bool(torch.isnan(O[seeing]).all()) and bool(torch.isnan(LSE[:, seeing]).all())
    rest = np.setdiff1d(np.arange(2 * T), [seeing])
    assert torch.equal(O[rest], clean[0][rest]) and torch.equal(LSE[:, rest], clean[1][:, rest])
