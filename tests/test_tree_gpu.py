"""Attention of drafted tokens over the paged cache, on the GPU, against the fp64 definition in
tests/cache_ref.py, which also derives the bounds.  Pages nobody owns and rows past a
sequence's end hold NaN throughout."""
import numpy as np
import pytest
import torch

from cache_ref import HALF_BF16, Batch, hold

pytestmark = pytest.mark.gpu


def _pkg():
    import online_softmax_flashattention_attention_gb300 as pkg
    return pkg


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def _run(batch, **more):
    args, kw = batch.dev()
    kw.update(more)
    O = torch.full_like(args[0], float("nan"))
    LSE = torch.full((args[0].shape[1], args[0].shape[0]), float("nan"), device="cuda")
    out = _pkg().attn_fwd_tree(*args, O, LSE, **kw)
    _pkg().cache_check()
    return out


CASES = [
    # hkv, G, page, ctx, T, masks
    (1, 1, 16, [0], [1], "chain"),
    (2, 4, 16, [0, 1, 15, 16, 17], [1, 1, 1, 1, 1], "chain"),
    (2, 8, 64, [63, 64, 65, 130], [1, 1, 1, 1], "tree"),
    (1, 16, 48, [47, 100], [1, 2], "tree"),
    (2, 3, 32, [0, 33, 500, 7], [5, 0, 3, 1], "tree"),
    (3, 5, 16, [200, 0, 3], [7, 4, 0], "random"),
    (1, 2, 128, [300, 40], [64, 63], "tree"),
    (2, 1, 16, [0, 0, 50], [64, 17, 16], "chain"),
    (1, 7, 256, [257, 511], [33, 9], "random"),
    (2, 2, 16, [0, 20], [3, 2], "none"),      # no drafted key visible: the first sequence's rows are empty
    (4, 32, 16, [31, 90], [1, 4], "tree"),
    (1, 1, 16, [1500], [1], "chain"),
    (1, 160, 16, [40], [2], "tree"),          # more heads a group than a tile has rows
    (1, 16, 32, [700, 90], [64, 41], "tree"),  # several tiles of one head, side by side
    (2, 9, 64, [300, 5, 0], [50, 29, 33], "random"),
]


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CASES)
def test_against_the_definition(case, d, f8):
    hkv, G, page, ctx, T, masks = case
    b = Batch(hash((d, page, G)) % 1000, hkv, G, d, page, f8, ctx, T, masks=masks)
    hold(*_run(b), b.reference())


@pytest.mark.parametrize("f8", [False, True])
def test_rows_outside_sequences_stay(f8):
    """Packed rows before and after the sequences, and past max_seqlen_q, are left as they were."""
    b = Batch(4, 2, 2, 64, 16, f8, [40, 3], [6, 2], gap=3, pad_q=4)
    O, LSE = _run(b)
    out = [0, 1, 2, 11, 12, 13, 14]
    assert bool(torch.isnan(O[out]).all()) and bool(torch.isnan(LSE[:, out]).all())
    refs = b.reference()
    live = slice(3, 11)
    hold(O[live], LSE[:, live], (refs[0][live], refs[1][:, live], refs[2][live], refs[3][:, live]))
    args, kw = b.dev()
    args[-1] = 4
    O2, LSE2 = torch.full_like(O, 7.0), torch.full_like(LSE, 7.0)
    _pkg().attn_fwd_tree(*args, O2, LSE2, **kw)
    _pkg().cache_check()
    assert bool((O2[7:9] == 7).all()) and bool((LSE2[:, 7:9] == 7).all())
    assert not bool((O2[3:7] == 7).all(-1).any())


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("G,T", [(2, 6), (8, 30)])
def test_nonfinite_values_reach_only_who_sees_them(f8, G, T):
    """NaN and infinities in K and V of drafted tokens: rows that do not see them are as if the
    tokens held anything else; rows that do are not finite where the formula is not."""
    ctx = 37
    for poison in (float("nan"), float("inf")):
        b = Batch(8, 2, G, 128, 16, f8, [ctx], [T])
        clean = _run(b)
        bad = [1, 4]
        for u in bad:
            pg, row = int(b.table[0][(ctx + u) // 16]), (ctx + u) % 16
            if f8:
                if poison != poison:
                    b.k.view(torch.uint8)[pg, :, row, 3] = 0x7F
                    b.v.view(torch.uint8)[pg, :, row, 100] = 0xFF
                else:
                    b.vs[pg, :, row] = 255  # an infinite scale
            else:
                b.k[pg, :, row, 3] = poison
                b.v[pg, :, row, 100] = poison
        O, LSE = _run(b)
        for i in range(T):
            see = [u for u in bad if (int(b.masks[i]) >> u) & 1]
            if not see:
                assert torch.equal(LSE[:, i], clean[1][:, i])
                # a slice that holds such a value is summed in fp32 instead of with bf16
                # probabilities: both lie within 2^-8 of the values' weighted size (up to 5 here)
                assert bool(((O[i] - clean[0][i]).float().abs() <= 4 * HALF_BF16 * 5).all())
            else:
                assert not bool(torch.isfinite(O[i, :, 100]).any())


@pytest.mark.parametrize("f8", [False, True])
def test_bad_pages_are_left_out(f8):
    """A context page outside the cache is masked and reported; a context longer than the table too."""
    pkg = _pkg()
    b = Batch(12, 2, 4, 64, 16, f8, [70], [2])
    args, kw = b.dev()
    table = args[3].clone()
    table[0, 1] = -1
    args[3] = table
    O, LSE = pkg.attn_fwd_tree(*args, **kw)
    with pytest.raises(pkg.AttnError) as e:
        pkg.cache_check()
    assert e.value.status == -9
    # the definition without positions 16 .. 31: the other pages, closed up
    c = Batch(12, 2, 4, 64, 16, f8, [70], [2])
    c.table = np.delete(c.table, 1, axis=1)
    c.ctx = [54]
    hold(O, LSE, c.reference())
    # a table with room for 32 of the 72 positions: the drafted tokens have no place at all
    args, kw = b.dev()
    args[3] = args[3][:, :2].contiguous()
    O, LSE = pkg.attn_fwd_tree(*args, **kw)
    with pytest.raises(pkg.AttnError):
        pkg.cache_check()
    c = Batch(12, 2, 4, 64, 16, f8, [70], [2])
    c.ctx, c.masks = [32], np.zeros(2, np.uint64)
    c.table = np.concatenate([c.table, c.table], axis=1)
    hold(O, LSE, c.reference())
    # no pages at all
    args, kw = b.dev()
    args[3] = args[3][:, :0].contiguous()
    O, LSE = pkg.attn_fwd_tree(*args, **kw)
    with pytest.raises(pkg.AttnError):
        pkg.cache_check()
    assert bool((O == 0).all()) and bool((LSE == -float("inf")).all())


def test_lengths_that_make_no_sense_are_clamped():
    """Negative contexts count as 0; cu_seqlens past the rows of Q end there."""
    pkg = _pkg()
    b = Batch(5, 1, 2, 64, 16, False, [0, 0], [3, 4])
    args, kw = b.dev()
    want = pkg.attn_fwd_tree(*args, **kw)
    args[4] = _i32([-9, -2 ** 31])
    args[5] = _i32([-3, 3, 900])
    got = pkg.attn_fwd_tree(*args, **kw)
    pkg.cache_check()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,hkv,G,T", [(300, 1, 2, 1), (3, 2, 4, 1), (9, 2, 2, 12), (1, 1, 1, 1), (2, 2, 8, 40), (150, 2, 4, 9)])
def test_long_ragged_batches_against_dense(B, hkv, G, T, d, f8):
    """Many CTAs a sequence and many sequences a CTA: all rows against a dense fp64 softmax over
    the rows read back from the cache (those are exact), under the same bounds."""
    pkg = _pkg()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(B * 1000 + d)
    r = np.random.default_rng(B + d)
    page = 32
    ctx = (r.integers(0, 60, B) if B > 100 else r.integers(2000, 9000, B)).tolist()
    n = [c + T for c in ctx]
    need = [-(-x // page) for x in n]
    P = sum(need) + 1
    table = np.zeros((B, max(need)), np.int64)
    perm, at = r.permutation(P), 0
    for b, x in enumerate(need):
        table[b, :x] = perm[at:at + x]
        at += x
    cu_k = np.concatenate([[0], np.cumsum(n)])
    cu_q = np.arange(B + 1) * T
    K, V = (torch.randn((int(cu_k[-1]), hkv, d), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    if f8:
        k, v = (torch.full((P, hkv, page, d), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
        sc = dict(k_scale=torch.full((P, hkv, page), 255, dtype=torch.uint8, device="cuda"))
        sc["v_scale"] = sc["k_scale"].clone()
    else:
        k, v = (torch.full((P, hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        sc = {}
    tab = _i32(table)
    pkg.attn_cache_write(K, V, k, v, tab, _i32(cu_k), **sc)
    K, V = pkg.attn_cache_read(k, v, tab, _i32(cu_k), int(cu_k[-1]), **sc)
    Q = torch.randn((B * T, hkv * G, d), generator=gen, device="cuda").to(torch.bfloat16)
    O, LSE = pkg.attn_fwd_tree(Q, k, v, tab, _i32(ctx), _i32(cu_q), T, **sc)
    pkg.cache_check()
    assert torch.equal(O, pkg.attn_fwd_tree(Q, k, v, tab, _i32(ctx), _i32(cu_q), T, **sc)[0])  # the same bits again
    for b in range(B) if B < 20 else r.integers(0, B, 40):
        Kb, Vb = K[cu_k[b]:cu_k[b + 1]].double(), V[cu_k[b]:cu_k[b + 1]].double()
        q = Q[b * T:(b + 1) * T].double().view(T, hkv, G, d)
        s = torch.einsum("thgd,nhd->thgn", q, Kb) / d ** 0.5
        vis = torch.arange(n[b], device="cuda")[None] <= ctx[b] + torch.arange(T, device="cuda")[:, None]
        s = s.masked_fill(~vis[:, None, None], -float("inf"))
        p = torch.softmax(s, -1)
        want = torch.einsum("thgn,nhd->thgd", p, Vb).reshape(T, hkv * G, d)
        A = torch.einsum("thgn,nhd->thgd", p, Vb.abs()).reshape(T, hkv * G, d)
        big = torch.einsum("thgd,nhd->thgn", q.abs(), Kb.abs()).amax() / d ** 0.5
        ds = d * 2.0 ** -24 * big + 2.0 ** -20
        if f8:  # query values under 2^-9 of the row's largest, as in cache_ref
            one = torch.exp2(torch.floor(torch.log2(q.abs().amax(-1, keepdim=True))))
            loss = torch.where(q.abs() < one * 2.0 ** -9, one * 2.0 ** -17, torch.zeros_like(q))
            ds = ds + torch.einsum("thgd,nhd->thgn", loss, Kb.abs()).amax() / d ** 0.5
        sums = (n[b] / 16 + 64) * 2.0 ** -24
        tol = HALF_BF16 * want.abs() + (HALF_BF16 + 4 * ds + 2 * sums) * 1.01 * A
        err = (O[b * T:(b + 1) * T].double() - want).abs()
        assert bool((err <= tol).all()), f"{float((err / tol).max()):.3g} of the bound"
        lse = torch.logsumexp(s, -1).reshape(T, hkv * G).t()
        assert bool(((LSE[:, b * T:(b + 1) * T].double() - lse).abs() <= ds + sums + 2.0 ** -17).all())


@pytest.mark.parametrize("f8", [False, True])
def test_attention_sinks_and_far_scores(f8):
    """One key that outweighs the rest by e^13 and 9000 keys that still matter together; scores
    that rise along the sequence, so that the running maximum moves in every block."""
    for kind in ("sink", "rising", "falling"):
        b = Batch(21, 1, 4, 64, 64, f8, [4000], [1], scale=1.0)
        q = torch.zeros_like(b.Q)
        q[..., 0] = 1.0
        b.Q = q
        for p in range(4001):
            pg, row = int(b.table[0][p // 64]), p % 64
            x = {"sink": 0.0 if p else 13.0, "rising": p / 64.0, "falling": (4000 - p) / 64.0}[kind]
            if f8:
                c = torch.zeros(64)
                c[0] = x
                b.k[pg, 0, row] = c.to(torch.float8_e4m3fn)
                b.ks[pg, 0, row] = 127
            else:
                b.k[pg, 0, row] = 0
                b.k[pg, 0, row, 0] = x
        hold(*_run(b), b.reference())


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("G,T", [(2, 5), (8, 20)])
def test_scales_far_apart(f8, G, T):
    """Keys whose values are 2^40 and more apart: a huge value that a row does not see, or sees with a
    weight of 2^-60, leaves the others what they are."""
    for kind in ("unseen", "weightless"):
        b = Batch(17, 1, G, 64, 16, f8, [90], [T], scale=1.0)
        if kind == "unseen":
            u = T - 1
            b.masks[: T - 1] &= np.uint64((1 << (T - 1)) - 1)
            b.masks[T - 1] = np.uint64((1 << (T - 1)) - 1)  # nobody sees the last token
            pos = 90 + u
        else:
            pos = 3
            b.Q[:, :, 0] = 1.0
        pg, row = int(b.table[0][pos // 16]), pos % 16
        if f8:
            b.vs[pg, :, row] = 230  # 2^103
            if kind == "weightless":
                c = torch.zeros(64)
                c[0] = -60.0
                b.k[pg, 0, row] = c.to(torch.float8_e4m3fn)
                b.ks[pg, :, row] = 127
        else:
            b.v[pg, :, row] = 2.0 ** 100
            if kind == "weightless":
                b.k[pg, 0, row] = 0
                b.k[pg, 0, row, 0] = -60.0
        hold(*_run(b), b.reference())


def test_two_threads_on_one_stream():
    """Calls of two host threads with the default workspace, launches interleaved."""
    import threading
    pkg = _pkg()
    a, b = Batch(31, 2, 4, 128, 16, True, [900, 30], [1, 1]), Batch(32, 2, 4, 128, 16, True, [12, 1500], [1, 1])
    calls = [x.dev() for x in (a, b)]
    wants = [pkg.attn_fwd_tree(*args, **kw) for args, kw in calls]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        args, kw = calls[i]
        for _ in range(200):
            O, LSE = pkg.attn_fwd_tree(*args, **kw)
            if not (torch.equal(O, wants[i][0]) and torch.equal(LSE, wants[i][1])):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    pkg.cache_check()
    assert not bad


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("G,T,d", [(1, 1, 64), (4, 1, 128), (8, 9, 64), (8, 9, 128)])
def test_a_wait_that_runs_out_is_reported(f8, G, T, d, monkeypatch):
    """A key block that is never loaded: every wait on it ends, the call reports a timeout, and the
    next call is right again."""
    pkg = _pkg()
    b = Batch(51, 2, G, d, 32, f8, [600, 200], [T, T])
    args, kw = b.dev()
    want = pkg.attn_fwd_tree(*args, **kw)
    pkg.cache_check()
    monkeypatch.setenv("ATTN_WAIT_LIMIT_MS", "20")
    monkeypatch.setenv("ATTN_ENABLE_TEST_HOOKS", "1")
    monkeypatch.setenv("ATTN_TEST_WITHHOLD_K_BLOCK", "1")
    pkg.attn_fwd_tree(*args, **kw)
    with pytest.raises(pkg.AttnError) as e:
        pkg.cache_check()
    assert e.value.status == -7
    monkeypatch.undo()
    got = pkg.attn_fwd_tree(*args, **kw)
    pkg.cache_check()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_capture_follows_the_lengths():
    """A captured call replayed with other contexts, tables and tree words, and two captured
    graphs with a workspace each on two streams at once."""
    pkg = _pkg()
    a, b = Batch(31, 2, 4, 128, 16, True, [700, 30], [1, 1]), Batch(32, 2, 4, 128, 16, True, [12, 500], [1, 1])
    graphs, outs, wants = [], [], []
    for x in (a, b):
        args, kw = x.dev()
        wants.append(pkg.attn_fwd_tree(*args, **kw))
        pkg.cache_check()
        args[4].zero_()  # captured with empty contexts
        O, LSE = torch.empty_like(args[0]), torch.empty_like(wants[-1][1])
        ws = torch.empty(pkg.tree_workspace_bytes(8, 2, 1, 128), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkg.attn_fwd_tree(*args, O, LSE, workspace=ws, **kw)
        args[4].copy_(_i32(x.ctx))
        graphs.append((graph, args, kw, ws))
        outs.append((O, LSE))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for (graph, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    pkg.cache_check()
    for got, want in zip(outs, wants):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_other_stream():
    pkg = _pkg()
    b = Batch(41, 2, 2, 64, 32, False, [400], [9])
    args, kw = b.dev()
    want = pkg.attn_fwd_tree(*args, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(50):
        O, LSE = pkg.attn_fwd_tree(*args, stream=side, **kw)
    side.synchronize()
    assert torch.equal(O, want[0]) and torch.equal(LSE, want[1])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("G,T", [(2, 3), (4, 20)])
def test_a_pool_without_pages(f8, G, T):
    """Nothing is cached and nothing can be: rows see nothing, and that is reported."""
    pkg = _pkg()
    k = torch.zeros((0, 2, 16, 64), dtype=torch.uint8 if f8 else torch.bfloat16, device="cuda")
    sc = {}
    if f8:
        k = k.view(torch.float8_e4m3fn)
        s = torch.zeros((0, 2, 16), dtype=torch.uint8, device="cuda")
        sc = dict(k_scale=s, v_scale=s)
    Q = torch.ones((2 * T, 2 * G, 64), dtype=torch.bfloat16, device="cuda")
    cu, ctx = _i32([0, T, 2 * T]), _i32([0, 70])
    for table in (_i32([[0, 1, 2], [3, -1, 7]]), torch.zeros((2, 0), dtype=torch.int32, device="cuda")):
        O, LSE = pkg.attn_fwd_tree(Q, k, k, table, ctx, cu, T, **sc)
        with pytest.raises(pkg.AttnError, match="no page"):
            pkg.cache_check()
        assert bool((O == 0).all()) and bool(torch.isneginf(LSE).all())
    pkg.cache_check()  # told once


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("T", [1, 40])
def test_output_in_the_query(f8, T):
    b = Batch(43, 2, 4, 128, 32, f8, [3000, 17, 0], [T, T, 1])
    args, kw = b.dev()
    want = _pkg().attn_fwd_tree(*args, **kw)
    O, _ = _pkg().attn_fwd_tree(*args, args[0], **kw)
    assert O is args[0] and torch.equal(O, want[0])


@pytest.mark.parametrize("f8", [False, True])
def test_decoding_run(f8):
    """As a program uses them: a prompt through the packed forward and into the cache, drafted
    trees appended and attended to, the prefix read back for a second prompt.  The forward over
    the rows read back is the yardstick for a chain's last token."""
    pkg = _pkg()
    H, d, page, lens, drafts = 4, 128, 32, [130, 61], [5, 3]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    new = lambda n: torch.randn((n, H, d), generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    total = sum(lens)
    Q, K, V = new(total), new(total), new(total)
    cu = _i32([0, 130, 191])
    k, v = (torch.zeros((12, H, page, d), dtype=torch.uint8 if f8 else torch.bfloat16, device="cuda") for _ in range(2))
    sc = {}
    if f8:
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        sc = dict(k_scale=torch.ones((12, H, page), dtype=torch.uint8, device="cuda"))
        sc["v_scale"] = sc["k_scale"].clone()
    table = _i32([[3, 9, 1, 7, 11], [0, 5, 2, 4, 6]])
    pkg.attn_fwd_varlen(Q, K, V, cu, cu, 130, causal=True)
    pkg.attn_cache_write(K, V, k, v, table, cu, **sc)
    cu_d, ctx = _i32([0, 5, 8]), _i32(lens)
    dq, dk, dv = new(8), new(8), new(8)
    pkg.attn_cache_write(dk, dv, k, v, table, cu_d, start_lens=ctx, **sc)
    O, LSE = pkg.attn_fwd_tree(dq, k, v, table, ctx, cu_d, 5, **sc)
    # the same tokens as a packed causal forward over the whole cache, read back
    cu_k = _i32([0, 135, 199])
    RK, RV = pkg.attn_cache_read(k, v, table, cu_k, 199, **sc)
    if not f8:
        assert torch.equal(RK[:130], K[:130]) and torch.equal(RK[130:135], dk[:5]) and torch.equal(RV[196:], dv[5:])
    O2, LSE2 = pkg.attn_fwd_varlen(dq, RK, RV, cu_d, cu_k, 5, causal=True)
    pkg.cache_check()
    # both round their probabilities and outputs to bf16; |v| < 6 here, e4m3 likewise
    assert bool(((O - O2).float().abs() <= 4 * HALF_BF16 * 6).all())
    assert bool(((LSE - LSE2).abs() <= 1e-4).all())
