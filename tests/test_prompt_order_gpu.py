"""attn_fwd_prompt where it takes tiles by cost (sequences of eight tiles and more), against fp64 on the GPU."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _pkg():
    import online_softmax_flashattention_attention_gb300 as pkg
    return pkg


def _cu(lens):
    return torch.as_tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()


def _hold(Q, K, V, nq, nk, O, LSE, poisoned=()):
    """Bounds as in test_many_sequences_and_items of the prompts' tests; poisoned: (sequence, key) whose value is NaN in
    column 5 of every head."""
    group = Q.shape[1] // K.shape[1]
    q0 = k0 = 0
    for b, (n, m) in enumerate(zip(nq, nk)):
        q, k, v = Q[q0:q0 + n].double(), *(x[k0:k0 + m].double().repeat_interleave(group, 1) for x in (K, V))
        bad = torch.zeros(n, dtype=torch.bool, device="cuda")
        for s, key in poisoned:
            if s == b:
                bad |= torch.arange(n, device="cuda") + m - n >= key
                v[key, :, 5] = 0
        z = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(Q.shape[2])
        z = z.masked_fill(torch.ones((n, m), dtype=torch.bool, device="cuda").triu(1 + m - n), -math.inf)
        p = torch.softmax(z, -1)
        want, size = torch.einsum("hij,jhd->ihd", p, v), torch.einsum("hij,jhd->ihd", p, v.abs())
        got = O[q0:q0 + n].double()
        if bad.any():
            assert torch.equal(torch.isnan(got[:, :, 5]), bad[:, None].expand(n, Q.shape[1]))
            got[bad, :, 5] = want[bad, :, 5]
        # the result's rounding and the probabilities' (2^-8 each), and 2^-12 for all in fp32
        assert bool(((got - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * size).all())
        assert bool(((LSE[:, q0:q0 + n].double() - torch.logsumexp(z, -1)).abs() <= 2.0 ** -15).all())
        q0, k0 = q0 + n, k0 + m


CASES = [
    # d, query heads, K/V heads, query lengths, keys before them
    (128, 16, 4, [1500, 900, 1, 0, 1025], [0, 0, 0, 0, 0]),
    (64, 4, 4, [1500, 900, 1, 0, 1025], [0, 0, 0, 0, 0]),
    (64, 32, 8, [1500, 900, 1, 0, 1025], [0, 0, 0, 0, 0]),
    (128, 32, 2, [1000, 200, 897], [300, 0, 128]),
    (64, 32, 2, [1000, 200, 897], [300, 0, 127]),
    (128, 32, 8, [1000, 40, 30, 20], [0, 3000, 2500, 2000]),   # by heads after all
    (64, 32, 8, [1000, 40, 30, 20], [0, 3000, 2500, 2000]),
    (128, 8, 2, [1100] + [17] * 100, [0] * 101),               # more sequences than are ranked by levels
    (64, 8, 2, [1100] + [17] * 95, [0] * 96),                  # as many as are
]


@pytest.mark.parametrize("case", CASES)
def test_against_definition(case):
    d, heads, kv, nq, before = case
    nk = [a + b for a, b in zip(nq, before)]
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    Q = torch.randn((sum(nq), heads, d), generator=g, device="cuda").to(torch.bfloat16)
    K, V = (torch.randn((sum(nk), kv, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    O, LSE = _pkg().attn_fwd_prompt(Q, K, V, _cu(nq), _cu(nk), max(nq))
    _pkg().status_sync()
    _hold(Q, K, V, nq, nk, O, LSE)
    if len(nq) < 10:  # the last key but one of the first sequence, one inside it, and the first of the last
        at = [(0, nk[0] - 2), (0, nk[0] // 2 + 3), (len(nq) - 1, 0)]
        starts = np.concatenate([[0], np.cumsum(nk)])
        for b, k in at:
            V[starts[b] + k, :, 5] = float("nan")
        O, LSE = _pkg().attn_fwd_prompt(Q, K, V, _cu(nq), _cu(nk), max(nq))
        _pkg().status_sync()
        _hold(Q, K, V, nq, nk, O, LSE, at)


@pytest.mark.parametrize("d,heads,kv,nq", [
    (128, 32, 8, [7000, 2100, 9000, 1500, 8000]),   # K and V past L2, by cost as lengths differ
    (128, 32, 8, [4200] * 6),                       # by heads as they do not
    (64, 32, 16, [7000, 2100, 9000, 1500, 8000]),
    (128, 8, 8, [12000, 9000, 6000]),               # a K/V head each: by heads
])
def test_past_l2(d, heads, kv, nq):
    """Whichever order the tiles go in: the rows of every sequence and head are those of the sequence alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(33)
    pkg, cu = _pkg(), _cu(nq)
    Q = torch.randn((sum(nq), heads, d), generator=g, device="cuda").to(torch.bfloat16)
    K, V = (torch.randn((sum(nq), kv, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    assert 2 * K.numel() * K.element_size() > 96 << 20
    O, LSE = pkg.attn_fwd_prompt(Q, K, V, cu, cu, max(nq))
    pkg.status_sync()
    q0 = 0
    for n in nq:
        at = slice(q0, q0 + n)
        one = _cu([n])
        want = pkg.attn_fwd_varlen(Q[at], *(x[at].repeat_interleave(heads // kv, 1) for x in (K, V)), one, one, n, causal=True)
        assert torch.equal(O[at], want[0]) and torch.equal(LSE[:, at], want[1])
        q0 += n


@pytest.mark.parametrize("d", [64, 128])
def test_without_causality_and_lies(d):
    """Not causal is not by cost; lengths past the rows, or fewer rows than max_seqlen_q, change nothing else."""
    g = torch.Generator(device="cuda")
    g.manual_seed(32)
    pkg = _pkg()
    Q = torch.randn((1300, 16, d), generator=g, device="cuda").to(torch.bfloat16)
    K, V = (torch.randn((1300, 4, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cu = _cu([1000, 300])
    O, LSE = pkg.attn_fwd_prompt(Q, K, V, cu, cu, 1000)
    for longest in (1300, 5000):
        got = pkg.attn_fwd_prompt(Q, K, V, cu, cu, longest)
        assert torch.equal(O, got[0]) and torch.equal(LSE, got[1])
    lie = torch.tensor([0, 1000, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    got = pkg.attn_fwd_prompt(Q, K, V, lie, lie, 1300)
    assert torch.equal(O, got[0]) and torch.equal(LSE, got[1])
    O2 = torch.zeros_like(O)
    pkg.attn_fwd_prompt(Q, K, V, cu, cu, 900, O2)  # a sequence's rows past max_seqlen_q may be left
    assert torch.equal(O2[:900], O[:900]) and torch.equal(O2[1000:], O[1000:])
    full = pkg.attn_fwd_prompt(Q, K, V, cu, cu, 1000, causal=False)
    same = pkg.attn_fwd_varlen(Q, K.repeat_interleave(4, 1), V.repeat_interleave(4, 1), cu, cu, 1000, causal=False)
    assert torch.equal(full[0], same[0]) and torch.equal(full[1], same[1])
