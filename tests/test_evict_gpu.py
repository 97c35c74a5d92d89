"""attn_cache_evict on the GPU: choice and packing have one right answer each."""
import numpy as np
import pytest
import torch

from prompt_ref import ref_evict

pytestmark = pytest.mark.gpu


def _pkg():
    import online_softmax_flashattention_attention_gb300 as pkg
    return pkg


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def _same(a, b):
    return np.array_equal(a, b, equal_nan=True)


def _pools(rng, P, hkv, page, d, f8):
    """Pools of distinct rows, as bytes, on the device."""
    if f8:
        k, v = (torch.from_numpy(rng.integers(0, 256, (P, hkv, page, d)).astype(np.uint8)).cuda() for _ in range(2))
        ks, vs = (torch.from_numpy(rng.integers(1, 248, (P, hkv, page)).astype(np.uint8)).cuda() for _ in range(2))
        return k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs
    k, v = (torch.from_numpy(rng.integers(-2 ** 15, 2 ** 15, (P, hkv, page, d)).astype(np.int16)).cuda().view(torch.bfloat16)
            for _ in range(2))
    return k, v, None, None


def _bits(t):
    if t is None:
        return None
    return (t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t).cpu().numpy()


def _weights(rng, shape, kind):
    w = rng.exponential(size=shape).astype(np.float32)
    if kind == "equal":
        w[:] = 0.25
    elif kind == "few":
        w = rng.integers(0, 3, shape).astype(np.float32)
    elif kind == "odd":  # every kind of number there is
        bits = rng.integers(0, 2 ** 32, shape, dtype=np.uint64).astype(np.uint32)
        w = bits.view(np.float32).copy()
        pick = rng.integers(0, 9, shape)
        for i, x in enumerate([np.nan, -np.inf, np.inf, 0.0, -0.0, 1e-45]):
            w[pick == i] = x
    elif kind == "close":  # neighbours in the last bits
        w = (0x3f800000 + rng.integers(0, 64, shape)).astype(np.uint32).view(np.float32).copy()
    return w


def _run(seed, hkv, d, page, f8, lens, keep, sink, recent, kind, other):
    pkg, rng = _pkg(), np.random.default_rng(seed)
    B = len(lens)
    need = [-(-n // page) for n in lens]
    room = -(-min(keep, max(max(need), 1) * page) // page)
    P = sum(need) + (B * room if other else 0) + 2
    order = rng.permutation(P)
    table = np.full((B, max(max(need), 1) + 1), 2 ** 31 - 1)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    to = order[at:at + B * room].reshape(B, room) if other else table
    k, v, ks, vs = _pools(rng, P, hkv, page, d, f8)
    w = _weights(rng, (P, hkv, page), kind)
    wd = torch.from_numpy(w).cuda()
    pools = [_bits(x) for x in (k, v, ks, vs)]
    kept_ref, lens_ref, new = ref_evict(pools, w, table, to, lens, keep, sink, recent, page)
    kept, out_lens = pkg.attn_cache_evict(k, v, wd, _i32(table), _i32(lens), keep, sink=sink, recent=recent,
                                          out_table=_i32(to) if other else None, k_scale=ks, v_scale=vs)
    pkg.cache_check()
    assert np.array_equal(kept.cpu().numpy(), kept_ref)
    assert np.array_equal(out_lens.cpu().numpy(), lens_ref)
    used = []
    for b in range(B):  # in place, rows past the kept ones mean nothing
        for i in range(int(lens_ref[b])):
            used.append((to[b, i // page], i % page))
    for got, want in zip([_bits(k), _bits(v), _bits(ks), _bits(vs), wd.cpu().numpy()], new):
        if want is None:
            continue
        if other:
            assert _same(got, want)
        else:
            assert _same(got, want)  # rows past the kept ones are left as they were, too


CASES = [
    # hkv, d, page, lengths, keep, sink, recent
    (1, 64, 16, [1], 1, 0, 0),
    (2, 128, 16, [40], 7, 1, 2),
    (8, 128, 64, [700, 63, 0, 64, 65, 500], 64, 4, 16),
    (3, 64, 48, [1000, 20], 999, 0, 0),
    (1, 128, 256, [5000], 1234, 100, 1000),
    (2, 64, 32, [300, 299], 100, 100, 0),
    (2, 64, 32, [300, 299], 100, 0, 100),
    (2, 128, 32, [300, 299], 100, 60, 40),
    (1, 64, 16, [2000] * 9, 1, 0, 0),
    (4, 128, 16, [50, 3], 60, 5, 5),
    (1, 128, 64, [20000], 3000, 3, 5),
]


@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_against_definition(case, f8, other):
    hkv, d, page, lens, keep, sink, recent = case
    _run(31, hkv, d, page, f8, lens, keep, sink, recent, "usual", other)


@pytest.mark.parametrize("kind", ["equal", "few", "odd", "close"])
@pytest.mark.parametrize("n,keep,sink,recent", [(500, 120, 0, 0), (9000, 4000, 7, 3), (70000, 1500, 0, 1)])
def test_weights_of_every_kind(kind, n, keep, sink, recent):
    _run(32, 2, 64, 64, True, [n, n // 3], keep, sink, recent, kind, False)
    _run(33, 1, 64, 128, False, [n], keep, sink, recent, kind, True)


def test_keep_nothing():
    _run(34, 2, 64, 16, False, [30, 0], 0, 0, 0, "usual", False)
    _run(34, 2, 64, 16, True, [30, 0], 0, 0, 0, "usual", True)


def test_more_keys_than_shared_memory_holds():
    """400000 positions and eight CTAs of 49152 keys: some weights are read again in every round."""
    pkg = _pkg()
    n, page, keep = 400001, 256, 70000
    P = -(-n // page)
    g = torch.Generator(device="cuda")
    g.manual_seed(35)
    k = torch.randint(0, 256, (P, 1, page, 64), generator=g, device="cuda", dtype=torch.uint8)
    v, ks = k.clone(), torch.randint(1, 200, (P, 1, page), generator=g, device="cuda", dtype=torch.uint8)
    w = torch.rand((P, 1, page), generator=g, device="cuda")
    w = (w * 50000).round()  # ties
    before = [x.clone() for x in (k, ks, w)]
    kept, lens = pkg.attn_cache_evict(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), w,
                                      torch.arange(P, dtype=torch.int32, device="cuda")[None], _i32([n]), keep, sink=11,
                                      recent=29, k_scale=ks, v_scale=ks.clone())
    pkg.cache_check()
    flat = before[2].view(-1)[11:n - 29]
    best = torch.sort(torch.sort(flat, descending=True, stable=True).indices[:keep - 40]).values + 11
    want = torch.cat((torch.arange(11, device="cuda"), best, torch.arange(n - 29, n, device="cuda")))
    assert torch.equal(kept.view(-1).long(), want) and int(lens) == keep
    assert torch.equal(k.view(-1, 64)[:keep], before[0].view(-1, 64)[want]) and torch.equal(v, k)
    assert torch.equal(ks.view(-1)[:keep], before[1].view(-1)[want]) and torch.equal(w.view(-1)[:keep], before[2].view(-1)[want])


@pytest.mark.parametrize("other", [False, True])
def test_long_sequence_many_slices(other):
    """One long sequence in bf16: columns (in place) or rows (other pages) shared by many blocks."""
    pkg = _pkg()
    n, page, keep, hkv, d = 40000, 64, 20000, 2, 128
    P = n // page
    g = torch.Generator(device="cuda")
    g.manual_seed(36)
    k, v = (torch.randn((2 * P, hkv, page, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.rand((2 * P, hkv, page), generator=g, device="cuda")
    table = torch.randperm(2 * P, generator=g, device="cuda").to(torch.int32).view(2, P)
    rows = lambda x, t: x[t.long()].transpose(0, 1).reshape((hkv, -1) + tuple(x.shape[3:]))  # noqa: E731
    before = [rows(x, table[0]) for x in (k, v, w)]
    to = table[1:] if other else None
    kept, lens = pkg.attn_cache_evict(k, v, w, table[:1].contiguous(), _i32([n]), keep, out_table=to)
    pkg.cache_check()
    for h in range(hkv):
        want = torch.sort(torch.sort(before[2][h], descending=True, stable=True).indices[:keep]).values
        assert torch.equal(kept[0, h].long(), want)
        for x, b in zip((k, v, w), before):
            assert torch.equal(rows(x, table[1 if other else 0])[h, :keep], b[h, want])


def test_bad_pages():
    """A missing page's positions count least and are packed as zeros; places without a page are not written."""
    pkg, rng = _pkg(), np.random.default_rng(37)
    k, v, ks, vs = _pools(rng, 8, 1, 16, 64, True)
    w = torch.from_numpy(rng.exponential(size=(8, 1, 16)).astype(np.float32)).cuda()
    w0 = w.clone()
    kept, lens = pkg.attn_cache_evict(k, v, w, _i32([[0, 99, 2]]), _i32([48]), 33, out_table=_i32([[5, -1, 6]]), k_scale=ks, v_scale=vs)
    with pytest.raises(pkg.AttnError, match="BAD_PAGE"):
        pkg.cache_check()
    assert kept[0, 0].tolist() == list(range(16)) + [16] + list(range(32, 48))
    assert torch.equal(w[5], w0[0]) and torch.equal(w[7], w0[7]) and float(w[6, 0, 0]) == float(w0[2, 0, 15])
    kept, lens = pkg.attn_cache_evict(k, v, w, _i32([[0, 1]]), _i32([1000]), 20, k_scale=ks, v_scale=vs)  # clamped
    pkg.cache_check()
    assert int(lens) == 20 and int(kept.max()) < 32


def test_captured_and_on_another_stream():
    pkg, rng = _pkg(), np.random.default_rng(38)
    k, v, _, _ = _pools(rng, 12, 2, 16, 64, False)
    w = torch.from_numpy(rng.exponential(size=(12, 2, 16)).astype(np.float32)).cuda()
    keep0 = [x.clone() for x in (k, v, w)]
    table, lens, to = _i32([[0, 1, 2, 3], [4, 5, 6, 7]]), _i32([64, 40]), _i32([[8, 9], [10, 11]])
    kept, out_lens = pkg.attn_cache_evict(k, v, w, table, lens, 20, out_table=to)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkg.attn_cache_evict(k, v, w, table, lens, 20, out_table=to, kept=kept, out_lens=out_lens)
    for n in ([10, 64], [64, 21]):
        for x, y in zip((k, v, w), keep0):
            x.copy_(y)
        lens.copy_(_i32(n))
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (k, v, w, kept, out_lens)]
        for x, y in zip((k, v, w), keep0):
            x.copy_(y)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        a, b = pkg.attn_cache_evict(k, v, w, table, lens, 20, out_table=to, stream=side)
        side.synchronize()
        for x, y in zip(got, (k, v, w, a, b)):
            assert torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x, y.view(torch.int16) if y.dtype == torch.bfloat16 else y)
