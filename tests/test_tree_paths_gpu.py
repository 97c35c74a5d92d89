"""Attention over the paged cache along paths the other files leave out: values that are not finite on both
sides of a block's and a piece's border, captured calls with the workspace the call makes for itself, the
128-row kernel captured and on two threads, offsets past 32 bits in both kernels and types."""
import threading

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


def _run(b):
    args, kw = b.dev()
    out = _pkg().attn_fwd_tree(*args, **kw)
    _pkg().cache_check()
    return [x.double().cpu().numpy() for x in out]


def _spoil(b, seq, node, kind, col):
    """Makes a drafted token's V not finite; returns the row's values [Hkv, d], zero where they are finite."""
    pos = b.ctx[seq] + node
    pg, row = int(b.table[seq][pos // b.page]), pos % b.page
    bad = np.zeros((b.hkv, b.d))
    if not b.f8:
        b.v[pg, :, row, col] = kind
        bad[:, col] = kind
    elif kind != kind:
        b.v.view(torch.uint8)[pg, :, row, col] = 0x7F
        bad[:, col] = np.nan
    else:  # an infinite scale: every value of the row, NaN where the code is 0
        b.vs[pg, :, row] = 255
        with np.errstate(invalid="ignore"):
            bad = b.v[pg, :, row].double().numpy() * np.inf
    return bad


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,G,T", [(2, 2, 6), (2, 4, 20), (1, 16, 64)])  # 16 rows; a tile; eight (two CTAs a key list)
@pytest.mark.parametrize("ctx", [[4090], [250] * 90])  # every unit shared by CTAs; mostly whole units
def test_nonfinite_values_across_borders(ctx, hkv, G, T, d, f8):
    """Drafted tokens on both sides of a multiple of 128 hold infinities of either sign and NaN in V: each
    row has what the formula gives for the tokens it sees, and nothing of the others."""
    if len(ctx) > 1 and T == 64:
        ctx = ctx[:12]
    b = Batch(91, hkv, G, d, 32, f8, ctx, [T] * len(ctx), masks="random")
    clean = _run(b)
    inf = float("inf")
    nodes = [(3, inf, 5), (4, -inf, 5), (T - 1, -inf, d - 1), (5 if T > 6 else 0, float("nan"), 33)]
    mine = sorted({0, len(ctx) // 2, len(ctx) - 1})
    bad = {(s, u): _spoil(b, s, u, kind, col) for s in mine for u, kind, col in nodes}
    O, LSE = _run(b)
    assert np.array_equal(LSE, clean[1])
    top = 4 * HALF_BF16 * b.v.float().abs().nan_to_num(0, 0, 0).max().item()
    if f8:
        top = 4 * HALF_BF16 * 6.0  # codes times scales: |v| < 6
    for s in range(len(ctx)):
        for i in range(T):
            row = b.cu[s] + i
            want = np.zeros((hkv, d))
            with np.errstate(invalid="ignore"):
                for u, _, _ in nodes:
                    if s in mine and (int(b.masks[row]) >> u) & 1:
                        want = want + np.where(np.isfinite(bad[s, u]), 0.0, bad[s, u])
            want = np.repeat(want, G, 0)
            got = O[row]
            assert np.array_equal(np.isnan(got), np.isnan(want))
            odd = np.isinf(want)
            assert np.array_equal(got[odd], want[odd])
            fine = np.isfinite(want)
            assert np.all(np.abs(got[fine] - clean[0][row][fine]) <= top)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("T", [1, 20])
def test_capture_with_the_workspace_of_the_call(f8, T):
    """Two captured calls without workspace=, in one graph, replayed with other lengths while eager calls and
    allocations go on."""
    pkg = _pkg()
    a, b = (Batch(s, 2, 4, 128, 16, f8, ctx, [T, T]) for s, ctx in ((33, [700, 30]), (34, [12, 1500])))
    calls = [x.dev() for x in (a, b)]
    wants = [pkg.attn_fwd_tree(*args, **kw) for args, kw in calls]
    pkg.cache_check()
    for args, _ in calls:
        args[4].zero_()  # captured with empty contexts
    outs = []
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for args, kw in calls:
            outs.append(pkg.attn_fwd_tree(*args, **kw))
    for x, (args, _) in zip((a, b), calls):
        args[4].copy_(_i32(x.ctx))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        graph.replay()
        junk = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(8)]
        args, kw = calls[0]
        eager = pkg.attn_fwd_tree(*args, **kw)
        other = pkg.attn_fwd_tree(*calls[1][0], stream=side, **calls[1][1])
        del junk
    torch.cuda.synchronize()
    pkg.cache_check()
    for got, want in list(zip(outs, wants)) + [(eager, wants[0]), (other, wants[1])]:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("f8", [False, True])
def test_tiles_captured_on_two_streams(f8):
    """Two graphs of the 128-row kernel, a workspace each, replayed at once with lengths set after capture."""
    pkg = _pkg()
    graphs, outs, wants = [], [], []
    for seed, ctx, T in ((35, [900, 3, 77], [20, 0, 9]), (36, [15, 2000, 0], [1, 33, 64])):
        x = Batch(seed, 2, 4, 128, 16, f8, ctx, T)
        args, kw = x.dev()
        args[6] = 64
        wants.append(pkg.attn_fwd_tree(*args, **kw))
        pkg.cache_check()
        args[4].zero_()
        O, LSE = torch.zeros_like(args[0]), torch.zeros_like(wants[-1][1])
        ws = torch.empty(pkg.tree_workspace_bytes(8, 2, 64, 128), dtype=torch.uint8, device="cuda")
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


@pytest.mark.parametrize("f8", [False, True])
def test_tiles_from_two_threads(f8):
    """The 128-row kernel called by two host threads on one stream, launches interleaved, and by both on
    streams of their own."""
    pkg = _pkg()
    calls = [Batch(s, 2, 4, 128, 16, f8, ctx, [20, 7]).dev() for s, ctx in ((37, [900, 30]), (38, [12, 1500]))]
    wants = [pkg.attn_fwd_tree(*args, **kw) for args, kw in calls]
    torch.cuda.synchronize()
    bad = []

    def work(i, own):
        args, kw = calls[i]
        stream = torch.cuda.Stream() if own else torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            for _ in range(100):
                O, LSE = pkg.attn_fwd_tree(*args, **kw)
                if not (torch.equal(O, wants[i][0]) and torch.equal(LSE, wants[i][1])):
                    bad.append(i)

    for own in (False, True):
        threads = [threading.Thread(target=work, args=(i, own)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    pkg.cache_check()
    assert not bad


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("T", [1, 9])
def test_offsets_past_32_bits(f8, T):
    """A pool of more than 2^31 elements, attended to on both sides of the border by one token and by more
    rows than a 16-row tile holds."""
    pkg = _pkg()
    hkv, G, d, page, P = 8, 4, 128, 1024, 2300  # 2300 * 8 * 1024 * 128 = 2.4e9
    k, v = (torch.empty((P, hkv, page, d), dtype=torch.uint8 if f8 else torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 31
    sc = {}
    if f8:
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        sc = {n: torch.empty((P, hkv, page), dtype=torch.uint8, device="cuda") for n in ("k_scale", "v_scale")}
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    n = 1500
    K, V = (torch.randn((n, hkv, d), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    table, cu = _i32([[P - 1, 1]]), _i32([0, n])
    pkg.attn_cache_write(K, V, k, v, table, cu, **sc)
    K2, V2 = pkg.attn_cache_read(k, v, table, cu, n, **sc)
    # what was written is where the table says, and reads back as half a step of e4m3 allows
    step = 2.0 ** -4 if f8 else 0.0
    for x, y in ((K, K2), (V, V2)):
        low = 2.0 ** -10 * x.float().abs().amax(-1, keepdim=True) / 224  # least code's half step, scale under max / 224
        assert bool(((x.float() - y.float()).abs() <= torch.maximum(step * x.float().abs(), step * 16 * low)).all())
    Q = torch.randn((T, hkv * G, d), generator=gen, device="cuda").to(torch.bfloat16)
    O, LSE = pkg.attn_fwd_tree(Q, k, v, table, _i32([n - T]), _i32([0, T]), T, **sc)
    pkg.cache_check()
    q = Q.double().view(T, hkv, G, d)
    s = torch.einsum("thgd,nhd->thgn", q, K2.double()) / d ** 0.5
    vis = torch.arange(n, device="cuda")[None] <= n - T + torch.arange(T, device="cuda")[:, None]
    s = s.masked_fill(~vis[:, None, None], -float("inf"))
    p = torch.softmax(s, -1)
    want = torch.einsum("thgn,nhd->thgd", p, V2.double()).reshape(T, hkv * G, d)
    A = torch.einsum("thgn,nhd->thgd", p, V2.double().abs()).reshape(T, hkv * G, d)
    lse = torch.logsumexp(s, -1).reshape(T, hkv * G).t()
    assert bool(((O.double() - want).abs() <= HALF_BF16 * want.abs() + 1.1 * HALF_BF16 * A).all())
    assert bool(((LSE.double() - lse).abs() <= 1e-3).all())
