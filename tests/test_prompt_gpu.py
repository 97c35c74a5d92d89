"""attn_fwd_prompt on the GPU against the definition in 64 bits."""
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


def _run(Q, K, V, cu_q, cu_k, max_q, **kw):
    O = torch.full(tuple(Q.shape), float("nan"), dtype=torch.bfloat16, device="cuda")
    LSE = torch.full((Q.shape[1], Q.shape[0]), float("nan"), device="cuda")
    pkg = _pkg()
    pkg.attn_fwd_prompt(Q.cuda(), K.cuda(), V.cuda(), _i32(cu_q), _i32(cu_k), max_q, O, LSE, **kw)
    pkg.status_sync()
    return O, LSE


CASES = [
    # Hkv, G, d, query lengths, keys before them, causal, gap, behind
    (1, 1, 128, [1], [0], True, 0, 0),
    (2, 4, 128, [77], [0], True, 0, 0),
    (1, 3, 64, [1, 2, 0, 127, 128, 129], [0, 0, 0, 0, 0, 0], True, 1, 5),
    (2, 2, 128, [130, 5, 257], [300, 0, 63], True, 0, 3),
    (1, 8, 64, [40, 1], [0, 500], True, 2, 0),
    (1, 7, 128, [33, 150], [95, 0], False, 0, 1),
    (3, 1, 64, [200, 64], [0, 1], False, 0, 0),
    (1, 2, 128, [200, 30], [-150, -30], True, 0, 2),   # fewer keys than queries: rows that see nothing
    (1, 5, 64, [140], [-139], True, 0, 0),
]


@pytest.mark.parametrize("joint", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_against_definition(case, joint):
    Hkv, G, d, nq, before, causal, gap, behind = case
    rng = np.random.default_rng(11)
    nk = [max(0, a + b) for a, b in zip(nq, before)]
    cu_q, cu_k = _cu(nq, gap), _cu(nk, gap + 1)
    tq, tk = cu_q[-1] + behind, cu_k[-1] + behind
    if joint:
        q = bf16(rng, (tq, Hkv * G + 2, d))
        kv = bf16(rng, (tk, 2 * Hkv + 1, d))
        Q, K, V = q[:, 1:1 + Hkv * G], kv[:, :Hkv], kv[:, Hkv:2 * Hkv]
    else:
        Q, K, V = bf16(rng, (tq, Hkv * G, d)), bf16(rng, (tk, Hkv, d)), bf16(rng, (tk, Hkv, d))
    K, V = K.clone() if not joint else K, V.clone() if not joint else V
    for t in (K, V):  # what no sequence owns holds anything
        t[:cu_k[0]] = float("nan")
        t[cu_k[-1]:] = float("inf")
    if joint:  # the device copies keep the strides
        q, kv = q.cuda(), kv.cuda()
        Qd, Kd, Vd = q[:, 1:1 + Hkv * G], kv[:, :Hkv], kv[:, Hkv:2 * Hkv]
    else:
        Qd, Kd, Vd = Q.cuda(), K.cuda(), V.cuda()
    scale = 1 / math.sqrt(d)
    O, LSE = _run(Qd, Kd, Vd, cu_q, cu_k, max(nq), causal=causal, scale=scale)
    hold_prompt(O, LSE, ref_prompt(f64(Q), f64(K), f64(V), cu_q, cu_k, scale, causal))


@pytest.mark.parametrize("d,heads", [(64, 4), (128, 4), (64, 64)])  # the last: two query tiles a CTA
@pytest.mark.parametrize("kind", ["nan", "inf", "both"])
@pytest.mark.parametrize("before", [0, 77])
def test_values_that_are_not_finite_stay_with_who_sees_them(d, heads, kind, before):
    """Infinities and NaN in keys and values of later tokens and of other sequences, diagonals in a block or across two."""
    rng = np.random.default_rng(12)
    nq = [260, 3, 129, 60]
    cu = _cu(nq)
    Q = bf16(rng, (cu[-1], heads, d))
    cu_k = _cu([n + before for n in nq])
    K, V = bf16(rng, (cu_k[-1], 2, d)), bf16(rng, (cu_k[-1], 2, d))
    bad = {"nan": [math.nan], "inf": [math.inf, -math.inf], "both": [math.nan, math.inf]}[kind]
    for i, row in enumerate((200, 259, 262, 263, 300, 390, 392, 440)):
        V[row, i % 2, 7 * i] = bad[i % len(bad)]
    K[255, 1] = math.nan
    K[391, 0] = math.nan
    O, LSE = _run(Q, K, V, cu, cu_k, max(nq))
    with np.errstate(invalid="ignore"):
        refs = ref_prompt(f64(Q), f64(K), f64(V), cu, cu_k, 1 / math.sqrt(d), True)
    hold_prompt(O, LSE, refs)


def test_query_that_is_not_finite():
    rng = np.random.default_rng(13)
    Q, K, V = bf16(rng, (150, 2, 128)), bf16(rng, (150, 1, 128)), bf16(rng, (150, 1, 128))
    Q[70, 0, 3] = math.nan
    O, LSE = _run(Q, K, V, [0, 150], [0, 150], 150)
    with np.errstate(invalid="ignore"):
        refs = ref_prompt(f64(Q), f64(K), f64(V), [0, 150], [0, 150], 1 / math.sqrt(128), True)
    assert np.isnan(refs[0][70, 0]).all()
    hold_prompt(O, LSE, refs)


@pytest.mark.parametrize("d", [64, 128])
def test_many_sequences_and_items(d):
    """More tiles than SMs, and more sequences than are ranked: every row of it, head by head in fp64 torch."""
    pkg = _pkg()
    g = torch.Generator(device="cuda")
    g.manual_seed(14)
    r = np.random.default_rng(14)
    for nq in (r.integers(0, 900, 40).tolist(), r.integers(0, 9, 700).tolist()):
        cu = _cu(nq)
        Q = torch.randn((cu[-1], 8, d), generator=g, device="cuda").to(torch.bfloat16)
        K, V = (torch.randn((cu[-1], 2, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        O, LSE = pkg.attn_fwd_prompt(Q, K, V, _i32(cu), _i32(cu), max(nq))
        pkg.status_sync()
        for b, n in enumerate(nq):
            at = slice(cu[b], cu[b + 1])
            k, v = (x[at].double().repeat_interleave(4, 1) for x in (K, V))
            z = torch.einsum("ihd,jhd->hij", Q[at].double(), k) / math.sqrt(d)
            z = z.masked_fill(torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1), -math.inf)
            p = torch.softmax(z, -1)
            want, size = torch.einsum("hij,jhd->ihd", p, v), torch.einsum("hij,jhd->ihd", p, v.abs())
            # the result's rounding and the probabilities' (2^-8 each), and 2^-12 for all in fp32
            assert bool(((O[at].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * size).all())
            assert bool(((LSE[:, at].double() - torch.logsumexp(z, -1)).abs() <= 2.0 ** -16).all())


@pytest.mark.parametrize("d", [64, 128])
def test_same_bits_as_the_packed_forward(d):
    """With a K/V head for every query head this is attn_fwd_varlen; with repeated heads too."""
    pkg, rng = _pkg(), np.random.default_rng(15)
    nq, nk = [300, 17, 128], [300, 400, 128]
    cu_q, cu_k = _i32(_cu(nq)), _i32(_cu(nk))
    Q = bf16(rng, (sum(nq), 4, d)).cuda()
    K, V = (bf16(rng, (sum(nk), 2, d)).cuda() for _ in range(2))
    O, LSE = pkg.attn_fwd_prompt(Q, K, V, cu_q, cu_k, 300)
    K4, V4 = (x.repeat_interleave(2, 1) for x in (K, V))
    for other in (pkg.attn_fwd_varlen(Q, K4, V4, cu_q, cu_k, 300, causal=True), pkg.attn_fwd_prompt(Q, K4, V4, cu_q, cu_k, 300)):
        assert torch.equal(O, other[0]) and torch.equal(LSE, other[1])


def test_outputs_with_strides_and_rows_left_alone():
    pkg, rng = _pkg(), np.random.default_rng(16)
    Q, K, V = bf16(rng, (100, 4, 64)).cuda(), bf16(rng, (100, 1, 64)).cuda(), bf16(rng, (100, 1, 64)).cuda()
    wide = torch.full((100, 7, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    cu = _i32([3, 40, 90])
    O, LSE = pkg.attn_fwd_prompt(Q, K, V, cu, cu, 50)
    pkg.attn_fwd_prompt(Q, K, V, cu, cu, 50, wide[:, 2:6, :64])
    pkg.status_sync()
    assert torch.equal(wide[3:90, 2:6, :64], O[3:90])
    wide[3:90, 2:6, :64] = 5.0
    assert (wide == 5.0).all()


def test_lengths_that_are_lies_stay_inside():
    """cu_seqlens past the rows there are is clamped; rows past max_seqlen_q are left as they were."""
    rng = np.random.default_rng(17)
    Q, K, V = bf16(rng, (64, 2, 128)), bf16(rng, (64, 1, 128)), bf16(rng, (64, 1, 128))
    O, LSE = _run(Q, K, V, [0, 30, 1000], [0, 30, 2 ** 31 - 1], 128)
    want = _run(Q, K, V, [0, 30, 64], [0, 30, 64], 64)
    assert torch.equal(O, want[0]) and torch.equal(LSE, want[1])
    Q, K, V = bf16(rng, (300, 2, 128)), bf16(rng, (300, 1, 128)), bf16(rng, (300, 1, 128))
    O, LSE = _run(Q, K, V, [0, 300], [0, 300], 128)
    assert torch.isfinite(O[:128]).all() and torch.isnan(O[128:]).all() and torch.isnan(LSE[:, 128:]).all()
    O, LSE = _run(Q, K, V, [-5, -3, -7, 300], [-1, 400, 5, 300], 300)  # anything at all ends inside the buffers


def test_captured_call_follows_the_lengths():
    pkg, rng = _pkg(), np.random.default_rng(18)
    Q, K, V = bf16(rng, (200, 4, 128)).cuda(), bf16(rng, (200, 2, 128)).cuda(), bf16(rng, (200, 2, 128)).cuda()
    cu = _i32([0, 100, 200])
    O, LSE = pkg.attn_fwd_prompt(Q, K, V, cu, cu, 200)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkg.attn_fwd_prompt(Q, K, V, cu, cu, 200, O, LSE)
    for c in ([0, 150, 200], [0, 0, 200], [0, 100, 200]):
        cu.copy_(_i32(c))
        g.replay()
        want = pkg.attn_fwd_prompt(Q, K, V, _i32(c), _i32(c), 200)
        torch.cuda.synchronize()
        assert torch.equal(O, want[0]) and torch.equal(LSE, want[1])


def test_no_keys_at_all():
    rng = np.random.default_rng(19)
    for total_k in (0, 4):
        Q, K = bf16(rng, (40, 2, 64)), bf16(rng, (total_k, 1, 64))
        O, LSE = _run(Q, K, K, [0, 40], [0, 0], 40)
        assert (O == 0).all() and torch.isneginf(LSE).all()
