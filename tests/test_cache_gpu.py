"""The paged cache on the GPU: written and read back exactly (its values have one right answer
each), against the definitions in tests/cache_ref.py."""
import numpy as np
import pytest
import torch

from cache_ref import Batch, ref_write

pytestmark = pytest.mark.gpu


def _pkg():
    import online_softmax_flashattention_attention_gb300 as pkg
    return pkg


def _same(a, b):
    """Equal values, NaN where NaN."""
    return np.array_equal(a, b, equal_nan=True)


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def _cache(P, hkv, page, d, f8, device="cuda"):
    """A pool filled with a value that no write makes here."""
    if f8:
        k, v = (torch.full((P, hkv, page, d), 0x55, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
                for _ in range(2))
        return k, v, *(torch.full((P, hkv, page), 9, dtype=torch.uint8, device=device) for _ in range(2))
    k, v = (torch.full((P, hkv, page, d), 77.0, dtype=torch.bfloat16, device=device) for _ in range(2))
    return k, v, None, None


def _tokens(seed, total, hkv, d, joint):
    r = np.random.default_rng(seed)
    x = torch.from_numpy(r.standard_normal((total, 2 * hkv + 3, d)).astype(np.float32)) * \
        torch.from_numpy(np.exp2(r.integers(-20, 20, (total, 2 * hkv + 3, 1))).astype(np.float32))
    x = x.to(torch.bfloat16)
    if joint:  # slices of one projection
        x = x.cuda()
        return x[:, 3:3 + hkv], x[:, 3 + hkv:]
    return x[:, :hkv].contiguous().cuda(), x[:, hkv:2 * hkv].contiguous().cuda()


WRITES = [
    # hkv, d, page, lengths, starts, joint
    (1, 64, 16, [1], [0], False),
    (8, 128, 64, [1, 1, 1, 1], [63, 64, 0, 200], True),
    (2, 128, 48, [0, 100, 0, 0, 7, 33], [5, 47, 1, 2, 0, 300], True),
    (3, 64, 32, [129, 1, 64], [0, 31, 95], False),
    (5, 128, 256, [300], [250], False),
    (1, 128, 16, [1] * 150, [3] * 150, False),
]


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("case", WRITES)
def test_write_and_read_back(case, f8):
    hkv, d, page, lens, start, joint = case
    pkg = _pkg()
    B = len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    need = [-(-(s + n) // page) for s, n in zip(start, lens)]
    P = sum(need) + 1
    perm = np.random.default_rng(7).permutation(P)
    table = np.full((B, max(need) + 1), -5)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    K, V = _tokens(11, cu[-1], hkv, d, joint)
    k, v, ks, vs = _cache(P, hkv, page, d, f8)
    want = [k.double().cpu().numpy(), v.double().cpu().numpy()] + \
        ([ks.cpu().numpy().astype(int), vs.cpu().numpy().astype(int)] if f8 else [None, None])
    ref_write(K.double().cpu().numpy(), V.double().cpu().numpy(), *want, table, cu, start, page)
    pkg.attn_cache_write(K, V, k, v, _i32(table), _i32(cu), start_lens=_i32(start), k_scale=ks, v_scale=vs)
    pkg.cache_check()
    for got, w in zip((k, v, ks, vs), want):
        if w is not None:
            assert _same(got.double().cpu().numpy(), w.astype(np.float64))
    # back: the same rows, as values
    RK, RV = pkg.attn_cache_read(k, v, _i32(table), _i32(cu), cu[-1], start_lens=_i32(start), k_scale=ks, v_scale=vs)
    pkg.cache_check()
    for out, c, s in ((RK, want[0], want[2]), (RV, want[1], want[3])):
        out = out.double().cpu().numpy()
        for b in range(B):
            for i in range(lens[b]):
                p = start[b] + i
                pg, row = table[b, p // page], p % page
                x = c[pg, :, row]
                if f8:
                    x = x * np.exp2(s[pg, :, row] - 127.0)[:, None]
                assert _same(out[cu[b] + i], x)


def test_write_special_values():
    """Rows of zeros, subnormals, the largest bf16, infinities, NaN, ties and the scale's border."""
    pkg = _pkg()
    d = 64
    rows = np.zeros((10, d), np.float32)
    rows[1] = 2.0 ** -133                              # the least bf16
    rows[2, 3] = 3.3895313892515355e38                 # the largest
    rows[3] = np.linspace(-1, 1, d)
    rows[3, 5], rows[3, 6], rows[3, 7] = np.inf, -np.inf, np.nan
    rows[4] = np.inf
    rows[5] = np.nan
    rows[6] = np.arange(d) * 0.5 + 200.0               # ties of the grid
    rows[6, 0] = 448.0
    rows[7] = 1.0
    rows[7, 0] = 450.0                                 # just past 448: the next power of two
    rows[8, ::2] = 2.0 ** -140                         # flushed to zero by bf16
    rows[9] = -(2.0 ** -126)
    x = torch.from_numpy(rows).to(torch.bfloat16)
    K = x[:, None, :].contiguous().cuda()
    k, v, ks, vs = _cache(1, 1, 16, d, True)
    want = [k.double().cpu().numpy(), v.double().cpu().numpy(), ks.cpu().numpy().astype(int), vs.cpu().numpy().astype(int)]
    ref_write(K.double().cpu().numpy(), K.double().cpu().numpy(), *want, [[0]], [0, 10], [0], 16)
    pkg.attn_cache_write(K, K, k, v, _i32([[0]]), _i32([0, 10]), k_scale=ks, v_scale=vs)
    pkg.cache_check()
    for got, w in zip((k, v, ks, vs), want):
        assert _same(got.double().cpu().numpy(), w.astype(np.float64))
    RK, _ = pkg.attn_cache_read(k, v, _i32([[0]]), _i32([0, 10]), 10, k_scale=ks, v_scale=vs)
    with np.errstate(invalid="ignore"):
        assert _same(RK.double().cpu().numpy()[:, 0], want[0][0, 0, :10] * np.exp2(want[2][0, 0, :10] - 127.0)[:, None])


@pytest.mark.parametrize("f8", [False, True])
def test_rows_outside_every_sequence_and_bad_pages(f8):
    """Packed rows before, between and after the sequences are not written and not read; a
    position without a page is left out, read as zeros, and reported once."""
    pkg = _pkg()
    hkv, d, page, P = 2, 128, 16, 4
    K, V = _tokens(3, 60, hkv, d, False)
    k, v, ks, vs = _cache(P, hkv, page, d, f8)
    before = [t.clone() for t in (k, v)]
    # sequence 0: rows 5..24 from position 10, pages 2, (bad); sequence 1: rows 25..44, pages 1, 3;
    # sequence 2: rows 45..49 at positions past the table
    table, cu, start = [[2, P], [1, 3], [0, -1]], [5, 25, 45, 50], [10, 0, 32]
    args = (_i32(table), _i32(cu))
    kw = dict(start_lens=_i32(start), k_scale=ks, v_scale=vs)
    pkg.attn_cache_write(K, V, k, v, *args, **kw)
    with pytest.raises(pkg.AttnError) as e:
        pkg.cache_check()
    assert e.value.status == -9
    pkg.cache_check()  # read once
    assert torch.equal(k[0].float(), before[0][0].float()) and torch.equal(v[0].float(), before[1][0].float())
    assert torch.equal(k[2, :, :10].float(), before[0][2, :, :10].float())
    if not f8:
        assert torch.equal(k[2, :, 10:], K[5:11].transpose(0, 1)) and torch.equal(v[3, :, :4], V[41:45].transpose(0, 1))
        assert torch.equal(k[3, :, 4:], before[0][3, :, 4:])
    RK, RV = (torch.full((60, hkv, d), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkg.attn_cache_read(k, v, *args, 60, RK, RV, **kw)
    with pytest.raises(pkg.AttnError):
        pkg.cache_check()
    for R in (RK, RV):
        assert bool((R[:5] == 5).all()) and bool((R[50:] == 5).all())
        assert bool((R[11:25] == 0).all()) and bool((R[45:50] == 0).all())
        assert not bool((R[5:11] == 5).all(-1).any()) and not bool((R[25:45] == 5).all(-1).any())
    # negative starts count as 0
    k2, v2, ks2, vs2 = _cache(P, hkv, page, d, f8)
    pkg.attn_cache_write(K[:3], V[:3], k2, v2, _i32([[1]]), _i32([0, 3]), start_lens=_i32([-7]), k_scale=ks2, v_scale=vs2)
    pkg.cache_check()
    k3, v3, ks3, vs3 = _cache(P, hkv, page, d, f8)
    pkg.attn_cache_write(K[:3], V[:3], k3, v3, _i32([[1]]), _i32([0, 3]), k_scale=ks3, v_scale=vs3)
    assert torch.equal(k2.float(), k3.float()) and torch.equal(v2.float(), v3.float())


def test_many_sequences_and_broadcast_heads():
    """5000 sequences, most of them empty; K and V with head stride 0 (one head for all)."""
    pkg = _pkg()
    r = np.random.default_rng(5)
    lens = (r.random(5000) < 0.05).astype(int) * r.integers(1, 4, 5000)
    cu = np.concatenate([[0], np.cumsum(lens)])
    total, page, d, hkv = int(cu[-1]), 16, 64, 4
    table = np.arange(5000)[:, None]
    x = torch.from_numpy(r.standard_normal((total, 1, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    K = x.expand(total, hkv, d)
    k, v, _, _ = _cache(5000, hkv, page, d, False)
    pkg.attn_cache_write(K, K, k, v, _i32(table), _i32(cu))
    pkg.cache_check()
    RK, RV = pkg.attn_cache_read(k, v, _i32(table), _i32(cu), total)
    assert torch.equal(RK, K) and torch.equal(RV, K)
    for b in np.nonzero(lens)[0][:40]:
        assert torch.equal(k[b, :, :lens[b]], K[cu[b]:cu[b + 1]].transpose(0, 1))


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements: pages on both sides of the border, written, read and
    attended to."""
    pkg = _pkg()
    hkv, d, page = 8, 128, 1024
    P = 2300  # 2300 * 8 * 1024 * 128 = 2.4e9 elements
    k = torch.empty((P, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 2 ** 31
    K, V = _tokens(1, 1500, hkv, d, False)
    K, V = (t.clamp(-4, 4) for t in (K, V))
    table, cu = _i32([[P - 1, 1]]), _i32([0, 1500])
    pkg.attn_cache_write(K, V, k, v, table, cu)
    RK, RV = pkg.attn_cache_read(k, v, table, cu, 1500)
    pkg.cache_check()
    assert torch.equal(RK, K) and torch.equal(RV, V)
    assert torch.equal(k[P - 1, :, :1024], K[:1024].transpose(0, 1)) and torch.equal(k[1, :, :476], K[1024:].transpose(0, 1))
    Q = torch.randn((1, hkv, d), device="cuda").to(torch.bfloat16)
    O, LSE = pkg.attn_fwd_tree(Q, k, v, table, _i32([1499]), _i32([0, 1]), 1)
    pkg.cache_check()
    s = torch.einsum("hd,nhd->hn", Q[0].double(), K.double()) / d ** 0.5
    want = torch.einsum("hn,nhd->hd", torch.softmax(s, -1), V.double())
    size = torch.einsum("hn,nhd->hd", torch.softmax(s, -1), V.double().abs())
    assert bool(((O[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1.2 * 2.0 ** -8 * size).all())
    assert bool(((LSE[:, 0].double() - torch.logsumexp(s, -1)).abs() <= 1e-3).all())


def test_other_stream_and_capture():
    """A write and a read captured once and replayed with other tokens and lengths."""
    pkg = _pkg()
    hkv, d, page = 4, 128, 32
    K, V = _tokens(2, 40, hkv, d, False)
    k, v, ks, vs = _cache(6, hkv, page, d, True)
    table, cu, start = _i32([[4, 0], [2, 5]]), _i32([0, 17, 40]), _i32([3, 20])
    kw = dict(start_lens=start, k_scale=ks, v_scale=vs)
    RK, RV = (torch.zeros((40, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step():
        pkg.attn_cache_write(K, V, k, v, table, cu, **kw)
        pkg.attn_cache_read(k, v, table, cu, 40, RK, RV, **kw)

    step()
    first = RK.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    K2, V2 = _tokens(9, 40, hkv, d, False)
    K.copy_(K2)
    V.copy_(V2)
    cu.copy_(_i32([0, 20, 40]))
    start.copy_(_i32([0, 11]))
    RK.zero_()
    graph.replay()
    pkg.cache_check()
    replayed = RK.clone()
    RK.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkg.attn_cache_write(K, V, k, v, table, cu, stream=side, **kw)
    pkg.attn_cache_read(k, v, table, cu, 40, RK, RV, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(RK, replayed) and not torch.equal(first, replayed)


def test_batch_helper_marks_what_nobody_owns():
    """The attention tests' pool really holds NaN outside the sequences."""
    b = Batch(1, 2, 1, 64, 16, True, [20], [3])
    own = 23
    assert int((b.k.view(torch.uint8)[:, 0, :, 0] != 0x7F).sum()) == own
