"""attn_fwd_prompt with its keys split (few tiles over many keys), against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

from prompt_ref import bf16, f64, hold_prompt, ref_prompt

pytestmark = pytest.mark.gpu


def _pkg():
    import online_softmax_flashattention_attention_gb300 as pkg
    return pkg


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def _cu(lens, gap=0):
    return (np.concatenate([[0], np.cumsum(lens)]) + gap).tolist()


def _run(Q, K, V, cu_q, cu_k, max_q, split=True, **kw):
    """In a workspace of 0xff bytes: whether states were written there is checked too."""
    pkg = _pkg()
    O = torch.full(tuple(Q.shape), float("nan"), dtype=torch.bfloat16, device="cuda")
    LSE = torch.full((Q.shape[1], Q.shape[0]), float("nan"), device="cuda")
    nbytes = pkg.prompt_workspace_bytes(len(cu_q) - 1, Q.shape[1], max_q, Q.shape[0], K.shape[0], Q.shape[2])
    assert nbytes > 0
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
    pkg.attn_fwd_prompt(Q.cuda(), K.cuda(), V.cuda(), _i32(cu_q), _i32(cu_k), max_q, O, LSE, workspace=ws, **kw)
    pkg.status_sync()
    assert bool((ws[1024:] != 255).any()) == split
    return O, LSE


CASES = [
    # Hkv, G, d, query lengths, keys before them, causal, gap, behind, whether keys are split
    (1, 4, 128, [100], [4000], True, 0, 0, True),
    (2, 2, 64, [130, 3], [3900, 0], True, 1, 5, True),
    (1, 8, 64, [1], [9000], True, 0, 0, True),
    (1, 2, 128, [70, 0, 5], [2500, 700, 1800], False, 2, 1, True),
    (4, 1, 64, [257], [5001], True, 0, 0, True),
    (1, 3, 128, [1, 128, 129, 40], [2047, 2048, 1, 6000], True, 0, 2, True),
    (1, 1, 128, [2300], [-400], True, 0, 0, True),      # rows that see nothing, tiles of them too
    (1, 1, 64, [2000], [0], True, 0, 0, True),
    (1, 2, 64, [20, 30, 40, 9, 8, 7, 6, 5], [620, 630, 640, 700, 700, 700, 700, 699], True, 0, 0, False),  # nothing is long
    (2, 2, 128, [0, 60, 0], [5000, 0, 900], True, 0, 0, False),    # what is long has no queries
]


@pytest.mark.parametrize("case", CASES)
def test_against_definition(case):
    Hkv, G, d, nq, before, causal, gap, behind, split = case
    rng = np.random.default_rng(21)
    nk = [max(0, a + b) for a, b in zip(nq, before)]
    cu_q, cu_k = _cu(nq, gap), _cu(nk, gap + 1)
    tq, tk = cu_q[-1] + behind, cu_k[-1] + behind
    Q, K, V = bf16(rng, (tq, Hkv * G, d)), bf16(rng, (tk, Hkv, d)), bf16(rng, (tk, Hkv, d))
    for t in (K, V):  # what no sequence owns holds anything
        t[:cu_k[0]] = float("nan")
        t[cu_k[-1]:] = float("inf")
    scale = 1 / math.sqrt(d)
    O, LSE = _run(Q, K, V, cu_q, cu_k, max(nq), split, causal=causal, scale=scale)
    hold_prompt(O, LSE, ref_prompt(f64(Q), f64(K), f64(V), cu_q, cu_k, scale, causal))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["nan", "inf", "both"])
def test_values_that_are_not_finite_stay_with_who_sees_them(d, kind):
    """In the prefix, on the diagonal's blocks (of two parts), in tokens that most rows do not see."""
    rng = np.random.default_rng(22)
    nq, before = [200, 60], [3000, 1750]
    cu, cu_k = _cu(nq), _cu([a + b for a, b in zip(nq, before)])
    Q, K, V = bf16(rng, (cu[-1], 2, d)), bf16(rng, (cu_k[-1], 2, d)), bf16(rng, (cu_k[-1], 2, d))
    bad = {"nan": [math.nan], "inf": [math.inf, -math.inf], "both": [math.nan, math.inf]}[kind]
    for i, row in enumerate((3001, 3070, 3073, 3150, 3199, 3200 + 1760, 3200 + 1800, 3200 + 700)):
        V[row, i % 2, 7 * i] = bad[i % len(bad)]
    K[3190, 1] = math.nan
    K[3200 + 1801, 0] = math.nan
    O, LSE = _run(Q, K, V, cu, cu_k, max(nq))
    with np.errstate(invalid="ignore"):
        refs = ref_prompt(f64(Q), f64(K), f64(V), cu, cu_k, 1 / math.sqrt(d), True)
    hold_prompt(O, LSE, refs)


def test_parts_of_very_different_size():
    """Scores of one part far above the others': their weights underflow."""
    rng = np.random.default_rng(23)
    Q, K, V = bf16(rng, (90, 2, 64)), bf16(rng, (4000, 1, 64)), bf16(rng, (4000, 1, 64))
    K[1000:1010] *= 300.0
    O, LSE = _run(Q, K, V, [0, 90], [0, 4000], 90)
    hold_prompt(O, LSE, ref_prompt(f64(Q), f64(K), f64(V), [0, 90], [0, 4000], 1 / 8, True))


def test_lengths_that_are_lies_stay_inside():
    rng = np.random.default_rng(24)
    Q, K, V = bf16(rng, (64, 2, 128)), bf16(rng, (4000, 1, 128)), bf16(rng, (4000, 1, 128))
    O, LSE = _run(Q, K, V, [0, 64], [0, 4000], 64)
    for cu_q, cu_k in (([0, 1000], [-9, 2 ** 31 - 1]), ([-7, 2 ** 31 - 1], [0, 4000])):
        got = _run(Q, K, V, cu_q, cu_k, 64)
        assert torch.equal(O, got[0]) and torch.equal(LSE, got[1])
    Q = bf16(rng, (300, 2, 128))
    O, LSE = _run(Q, K, V, [0, 300], [0, 4000], 128)  # rows past max_seqlen_q are left as they were
    assert torch.isfinite(O[:128]).all() and torch.isnan(O[128:]).all() and torch.isnan(LSE[:, 128:]).all()
    _run(Q, K, V, [-5, -3, -7, 300], [-1, 4400, 5, 300], 300, False)  # anything at all ends inside the buffers


def test_captured_calls_and_streams():
    """Two graphs that run at once have workspaces of their own; so have two streams; lengths may change."""
    pkg, rng = _pkg(), np.random.default_rng(25)
    Q, K, V = bf16(rng, (100, 4, 128)).cuda(), bf16(rng, (6000, 2, 128)).cuda(), bf16(rng, (6000, 2, 128)).cuda()
    cuts = [_i32([0, 40, 100]) for _ in range(2)], [_i32([0, 3000, 6000]), _i32([0, 5500, 6000])]
    wants = [[x.clone() for x in pkg.attn_fwd_prompt(Q, K, V, a, b, 100)] for a, b in zip(*cuts)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a, b in zip(*cuts):
        O, LSE = torch.zeros_like(Q), torch.zeros((4, 100), device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkg.attn_fwd_prompt(Q, K, V, a, b, 100, O, LSE)
        graphs.append(g)
        outs.append((O, LSE))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, wants):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = [[pkg.attn_fwd_prompt(Q, K, V, a, b, 100, stream=s) for a, b, s in zip(*cuts, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for row in got:
        for one, want in zip(row, wants):
            assert torch.equal(one[0], want[0]) and torch.equal(one[1], want[1])
    cuts[1][0].copy_(cuts[1][1])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], wants[1][0]) and torch.equal(outs[0][1], wants[1][1])


def test_refusals():
    pkg, rng = _pkg(), np.random.default_rng(26)
    Q, K, V = bf16(rng, (100, 4, 128)).cuda(), bf16(rng, (6000, 2, 128)).cuda(), bf16(rng, (6000, 2, 128)).cuda()
    cu_q, cu_k = _i32([0, 100]), _i32([0, 6000])
    nbytes = pkg.prompt_workspace_bytes(1, 4, 100, 100, 6000, 128)
    ws = torch.empty(nbytes + 16, dtype=torch.uint8, device="cuda")
    for bad in (ws[:nbytes - 1], ws[8:nbytes + 8]):
        with pytest.raises(RuntimeError):
            pkg.attn_fwd_prompt(Q, K, V, cu_q, cu_k, 100, workspace=bad)
    for bad in (ws.cpu(), ws[::2], ws.view(torch.float32)):
        with pytest.raises(ValueError):
            pkg.attn_fwd_prompt(Q, K, V, cu_q, cu_k, 100, workspace=bad)
    assert pkg.prompt_workspace_bytes(0, 4, 100, 100, 6000, 128) == 0 and pkg.prompt_workspace_bytes(1, 4, 100, 100, 6000, 96) == 0
    assert pkg.prompt_workspace_bytes(1, 32, 10000, 10000, 10000, 128) == 0  # tiles enough
