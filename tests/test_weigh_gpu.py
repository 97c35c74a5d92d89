"""attn_cache_weigh on the GPU against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

from cache_ref import Batch
from prompt_ref import f64, ref_weigh

pytestmark = pytest.mark.gpu


def _pkg():
    import online_softmax_flashattention_attention_gb300 as pkg
    return pkg


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def _lse(bt):
    """fp32 LSE of a batch's chains, -inf outside every sequence."""
    total, Hq, d = bt.Q.shape
    q, k = f64(bt.Q), f64(bt.k)
    ks = None if bt.ks is None else bt.ks.numpy()
    from cache_ref import rows_of
    out = np.full((Hq, total), -np.inf)
    for b in range(len(bt.ctx)):
        n = bt.ctx[b] + bt.T[b]
        K = rows_of(k, ks, bt.table, b, n, bt.page)
        see = np.arange(n)[None] <= bt.ctx[b] + np.arange(bt.T[b])[:, None]
        for h in range(Hq if bt.T[b] else 0):
            s = np.where(see, bt.scale * (q[bt.cu[b]:bt.cu[b + 1], h] @ K[:, h // bt.G].T), -np.inf)
            m = s.max(1)
            out[h, bt.cu[b]:bt.cu[b + 1]] = m + np.log(np.exp(s - m[:, None]).sum(1))
    return out.astype(np.float32)


def _check(bt, decay, in_place=False, lse=None, seed=1):
    pkg, rng = _pkg(), np.random.default_rng(seed)
    shape = tuple(bt.k.shape[:3])
    w = rng.exponential(size=shape).astype(np.float32)
    own = np.zeros(shape, bool)  # what is no sequence's, and (decay) what the call brings, holds NaN
    for b in range(len(bt.ctx)):
        for p in range(bt.ctx[b] if bt.T[b] else 0):
            own[bt.table[b, p // bt.page], :, p % bt.page] = True
    w[~own] = np.nan
    lse = _lse(bt) if lse is None else lse
    out = w.copy() if in_place else np.full(shape, -3.0, np.float32)
    args = bt.dev()[0]
    Wd = torch.from_numpy(w).cuda()
    Od = Wd if in_place else torch.from_numpy(out).cuda()
    kw = {} if bt.ks is None else {"k_scale": bt.ks.cuda()}
    got = pkg.attn_cache_weigh(args[0], torch.from_numpy(lse).cuda(), args[1], None if decay == 0 and not in_place else Wd, args[3],
                               args[4], args[5], None if in_place else Od, decay=decay, scale=bt.scale, **kw)
    pkg.cache_check()
    assert got is Od
    want, tol = ref_weigh(f64(bt.Q), lse.astype(np.float64), f64(bt.k), None if bt.ks is None else bt.ks.numpy(), bt.table, bt.ctx,
                          bt.cu, bt.page, bt.scale, decay, w.astype(np.float64), out.astype(np.float64))
    g = f64(got)
    assert np.array_equal(np.isnan(g), np.isnan(want))
    ok = ~np.isnan(want)
    worst = np.max(np.abs(g[ok] - want[ok]) - tol[ok])
    assert worst <= 0, f"{np.nanmax(np.abs(g[ok] - want[ok]) / np.maximum(tol[ok], 1e-300)):.3g} of the bound"
    return g


CASES = [
    # hkv, G, d, page, ctx, T, extras
    (1, 1, 64, 16, [0], [1], {}),
    (8, 4, 128, 16, [517], [1], {}),
    (2, 4, 128, 64, [0, 300, 127, 128], [1, 1, 0, 1], dict(pad_q=3, gap=2)),
    (1, 7, 64, 48, [130, 0], [5, 19], {}),
    (2, 3, 128, 32, [1, 255, 40], [130, 2, 0], dict(gap=1)),
    (1, 8, 128, 256, [0], [150], {}),
    (3, 1, 64, 128, [10, 0, 700], [300, 129, 1], dict(pad_q=40)),
    (1, 5, 64, 16, [3] * 70, [1, 0] * 35, {}),
    (1, 33, 128, 16, [100], [9], {}),
    (1, 200, 64, 16, [60], [3], {}),
]


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_against_definition(case, f8):
    hkv, G, d, page, ctx, T, more = case
    bt = Batch(21, hkv, G, d, page, f8, ctx, T, masks="chain", **more)
    bt.Q[:bt.cu[0]] = float("nan")   # rows of no sequence
    bt.Q[bt.cu[-1]:] = float("inf")
    _check(bt, 0.9)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("decay", [0.0, 1.0, -0.5])
def test_decay_and_place(decay, f8):
    bt = Batch(22, 2, 4, 128, 32, f8, [200, 0, 33], [3, 70, 1], masks="chain")
    a = _check(bt, decay)
    b = _check(bt, decay, in_place=True)
    own = np.isfinite(b) & (a != -3.0)
    assert np.array_equal(a[own], b[own])


@pytest.mark.parametrize("f8", [False, True])
def test_far_scores_and_rows_that_saw_nothing(f8):
    """Large scores (an LSE of hundreds); rows whose LSE is -inf add nothing; NaN stays with who sees it."""
    bt = Batch(23, 1, 2, 64, 16, f8, [90], [40], masks="chain", scale=40.0)
    lse = _lse(bt)
    assert np.abs(lse).max() > 300
    lse[0, 5] = lse[1, 17] = -np.inf
    _check(bt, 1.0, lse=lse)
    bt.Q[20, 1, 3] = float("nan")
    lse[1, 20] = np.nan
    g = _check_nan(bt, lse, 90 + 20)


def _check_nan(bt, lse, last):
    pkg = _pkg()
    out = torch.zeros(tuple(bt.k.shape[:3]), device="cuda")
    args = bt.dev()[0]
    kw = {} if bt.ks is None else {"k_scale": bt.ks.cuda()}
    pkg.attn_cache_weigh(args[0], torch.from_numpy(lse).cuda(), args[1], None, args[3], args[4], args[5], out, decay=0.0,
                         scale=bt.scale, **kw)
    pkg.cache_check()
    for p in range(bt.ctx[0] + bt.T[0]):
        assert math.isnan(float(out[int(bt.table[0, p // bt.page]), 0, p % bt.page])) == (p <= last)


def test_keys_that_are_not_finite_stay_alone():
    bt = Batch(24, 1, 4, 128, 16, False, [200], [30], masks="chain")
    lse = _lse(bt)
    bad = {5: float("nan"), 100: float("inf"), 215: float("nan")}
    for p, x in bad.items():
        bt.k[int(bt.table[0, p // 16]), 0, p % 16, 7] = x
    pkg, args = _pkg(), bt.dev()[0]
    out = torch.zeros(tuple(bt.k.shape[:3]), device="cuda")
    pkg.attn_cache_weigh(args[0], torch.from_numpy(lse).cuda(), args[1], None, args[3], args[4], args[5], out, decay=0.0)
    pkg.cache_check()
    for p in range(230):
        v = float(out[int(bt.table[0, p // 16]), 0, p % 16])
        assert math.isfinite(v) == (p not in bad)


@pytest.mark.parametrize("f8", [False, True])
def test_large_prompt_against_torch(f8):
    """A whole prompt and a long context, in fp64 torch, and the same bits a second time and in another batch."""
    pkg = _pkg()
    g = torch.Generator(device="cuda")
    g.manual_seed(25)
    for hkv, G, d, ctx, T in ((2, 4, 128, 0, 2500), (4, 2, 64, 30000, 3), (1, 8, 128, 1000, 600)):
        n, page = ctx + T, 64
        P = -(-n // page)
        K = torch.randn((n, hkv, d), generator=g, device="cuda").to(torch.bfloat16)
        k, v = (torch.zeros((P + 2, hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        kw = {}
        if f8:
            k, v = (torch.zeros((P + 2, hkv, page, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
            kw = {"k_scale": torch.ones((P + 2, hkv, page), dtype=torch.uint8, device="cuda")}
            kw["v_scale"] = torch.ones_like(kw["k_scale"])
        table = torch.randperm(P + 2, generator=g, device="cuda")[:P].to(torch.int32)[None].contiguous()
        pkg.attn_cache_write(K, K, k, v, table, _i32([0, n]), **kw)
        K = pkg.attn_cache_read(k, v, table, _i32([0, n]), n, **kw)[0]
        kw.pop("v_scale", None)
        Q = torch.randn((T, hkv * G, d), generator=g, device="cuda").to(torch.bfloat16)
        z = torch.einsum("thd,nhd->htn", Q.double(), K.double().repeat_interleave(G, 1)) / math.sqrt(d)
        see = torch.arange(n, device="cuda")[None] <= ctx + torch.arange(T, device="cuda")[:, None]
        z = z.masked_fill(~see, -math.inf)
        LSE = torch.logsumexp(z, -1).float()
        want = torch.exp(z - LSE.double()[..., None]).view(hkv, G * T, n).sum(1)
        out = torch.zeros((P + 2, hkv, page), device="cuda")
        args = (Q, LSE, k, None, table, _i32([ctx]), _i32([0, T]), out)
        pkg.attn_cache_weigh(*args, decay=0.0, **kw)
        pkg.cache_check()
        got = out[table[0].long()].transpose(0, 1).reshape(hkv, -1)[:, :n].double()
        # fp32 scores of d products (d u times sum |q k| <= 6 d u in sigmas of its mean size), exponents and sums
        assert bool(((got - want).abs() <= want * 2.0 ** -14 + 1e-30).all())
        again = torch.zeros_like(out)
        pkg.attn_cache_weigh(*args[:-1], again, decay=0.0, **kw)
        two = torch.zeros_like(out)  # the same sequence behind an empty one, in a batch with another head count of tokens
        pkg.attn_cache_weigh(Q, LSE, k, None, table.repeat(2, 1), _i32([0, ctx]), _i32([0, 0, T]), two, decay=0.0, **kw)
        assert torch.equal(out, again) and torch.equal(out, two)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("hkv,G,d,page,B,ctx,T", [
    (8, 4, 128, 64, 48, (2000, 5000), (1, 1)),      # long units, one step after the other
    (8, 4, 64, 48, 60, (3000, 4500), (0, 3)),
    (4, 5, 128, 16, 70, (0, 9000), (1, 20)),
    (8, 1, 64, 128, 300, (0, 400), (1, 1)),          # many short ones
    (2, 4, 128, 32, 40, (0, 2000), (1, 300)),        # one tile here, several there
])
def test_batches_against_torch(hkv, G, d, page, B, ctx, T, f8):
    """Batches that go round the SMs several times, every key of them, in fp64 torch."""
    pkg, r = _pkg(), np.random.default_rng(29)
    g = torch.Generator(device="cuda")
    g.manual_seed(29)
    ctxs, Ts = r.integers(ctx[0], ctx[1] + 1, B), r.integers(T[0], T[1] + 1, B)
    need = [-(-int(c + t) // page) for c, t in zip(ctxs, Ts)]
    P = sum(need) + 1
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((B, max(need)), dtype=torch.int32, device="cuda")
    for b in range(B):
        table[b, :need[b]] = order[sum(need[:b]):sum(need[:b + 1])]
    k = torch.randn((P, hkv, page, d), generator=g, device="cuda").to(torch.bfloat16)
    kw, kd = {}, k.double()
    if f8:
        codes = k.float().clamp(-4, 4).to(torch.float8_e4m3fn)
        s = torch.randint(125, 130, (P, hkv, page), generator=g, device="cuda", dtype=torch.uint8)
        kd = codes.double() * torch.exp2(s.double() - 127)[..., None]
        k, kw = codes, {"k_scale": s}
    cu = np.concatenate([[0], np.cumsum(Ts)])
    total = int(cu[-1])
    Q = torch.randn((total, hkv * G, d), generator=g, device="cuda").to(torch.bfloat16)
    LSE = torch.full((hkv * G, total), -math.inf, device="cuda")
    w = torch.rand((P, hkv, page), generator=g, device="cuda")
    want, tol = torch.full((P, hkv, page), -5.0, dtype=torch.float64, device="cuda"), torch.zeros((P, hkv, page), device="cuda")
    for b in range(B):
        c, t = int(ctxs[b]), int(Ts[b])
        if t == 0:
            continue
        p = torch.arange(c + t, device="cuda")
        pg, row = table[b].long()[p // page], p % page
        K = kd[pg, :, row].transpose(0, 1)
        q = Q[cu[b]:cu[b + 1]].double().view(t, hkv, G, d).permute(1, 2, 0, 3).reshape(hkv, G * t, d)
        z = q @ K.transpose(1, 2) / math.sqrt(d)
        see = (p[None] <= c + torch.arange(t, device="cuda")[:, None]).repeat(G, 1)
        z = z.masked_fill(~see, -math.inf)
        lse = torch.logsumexp(z, -1).float()
        LSE[:, cu[b]:cu[b + 1]] = lse.view(hkv * G, t)
        prob = torch.exp(z - lse.double()[..., None])
        old = torch.where(p < c, 0.5 * w[pg, :, row].double().t(), 0.0)
        want[pg, :, row] = (old + prob.sum(1)).t()
        # B of the module's bounds, and an e4m3 query's 2^-17 of its row's largest value
        big = (q.abs() @ K.abs().transpose(1, 2)) / math.sqrt(d)
        lost = (q.abs().amax(-1, keepdim=True) * 2.0 ** -17 * K.abs().sum(-1)[:, None]) / math.sqrt(d) if f8 else 0.0
        e = prob * ((d + 16) * 2.0 ** -24 * (big + lse.abs()[..., None]) + lost + 2.0 ** -21 * (z.abs().nan_to_num(posinf=0.0) + lse.abs()[..., None] + 1))
        tol[pg, :, row] = (e.sum(1) + (t * G / 4 + 64) * 2.0 ** -24 * prob.sum(1) + 2.0 ** -22 * old).t().float() + 1e-30
    out = torch.full((P, hkv, page), -5.0, device="cuda")
    pkg.attn_cache_weigh(Q, LSE, k, w, table, _i32(ctxs), _i32(cu), out, decay=0.5, **kw)
    pkg.cache_check()
    assert bool(((out.double() - want).abs() <= 1.01 * tol).all())


def test_bad_pages_are_reported_and_left_out():
    pkg = _pkg()
    bt = Batch(26, 2, 2, 64, 16, False, [50], [4], masks="chain")
    lse = torch.from_numpy(_lse(bt)).cuda()
    args = bt.dev()[0]
    out = torch.zeros(tuple(bt.k.shape[:3]), device="cuda")
    pkg.attn_cache_weigh(args[0], lse, args[1], None, args[3], args[4], args[5], out, decay=0.0)
    pkg.cache_check()
    table = args[3].clone()
    table[0, 1] = -1
    table[0, 2] = args[1].shape[0]
    got = torch.full_like(out, 9.0)
    pkg.attn_cache_weigh(args[0], lse, args[1], None, table, args[4], args[5], got, decay=0.0)
    with pytest.raises(pkg.AttnError, match="BAD_PAGE"):
        pkg.cache_check()
    for s in (0, 3):
        pg = int(args[3][0, s])
        last = 54 - 16 * s
        assert torch.equal(got[pg, :, :last], out[pg, :, :last])
    assert (got[args[3][0, 1:3].long()] == 9.0).all()
    got.fill_(9.0)  # a table without room for the last tokens
    pkg.attn_cache_weigh(args[0], lse, args[1], None, args[3][:, :2].contiguous(), args[4], args[5], got, decay=0.0)
    with pytest.raises(pkg.AttnError, match="BAD_PAGE"):
        pkg.cache_check()
    assert torch.equal(got[args[3][0, 0].long()], out[args[3][0, 0].long()])


def test_captured_call_follows_the_lengths():
    pkg = _pkg()
    a = Batch(27, 2, 4, 128, 16, True, [100, 30], [2, 3], masks="chain")
    b = Batch(27, 2, 4, 128, 16, True, [20, 110], [4, 1], masks="chain")
    dev = a.dev()[0]
    pages = max(a.k.shape[0], b.k.shape[0])
    k = torch.zeros((pages,) + tuple(a.k.shape[1:]), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ks = torch.ones((pages, 2, 16), dtype=torch.uint8, device="cuda")
    wide = max(a.max_pages, b.max_pages)
    table = torch.zeros((2, wide), dtype=torch.int32, device="cuda")
    lse = torch.zeros((8, 5), device="cuda")
    out = torch.zeros((pages, 2, 16), device="cuda")
    args = (dev[0], lse, k, None, table, dev[4], dev[5], out)

    def fill(bt):
        k.view(torch.uint8)[:bt.k.shape[0]] = bt.k.cuda().view(torch.uint8)
        ks[:bt.k.shape[0]] = bt.ks.cuda()
        t = np.full((2, wide), -1)
        t[:, :bt.max_pages] = np.where(bt.table < 2 ** 31 - 1, bt.table, -1)
        table.copy_(_i32(t))
        dev[0].copy_(bt.Q.cuda())
        dev[4].copy_(_i32(bt.ctx))
        dev[5].copy_(_i32(bt.cu))
        lse.copy_(torch.from_numpy(_lse(bt)).cuda())

    fill(a)
    pkg.attn_cache_weigh(*args, decay=0.0, k_scale=ks)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkg.attn_cache_weigh(*args, decay=0.0, k_scale=ks)
    for bt in (b, a):
        fill(bt)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.zero_()
        pkg.attn_cache_weigh(*args, decay=0.0, k_scale=ks)
        pkg.cache_check()
        assert torch.equal(got, out) and float(out.abs().sum()) > 0


def test_pools_past_32_bits():
    """Keys and weights at offsets past 2^31 elements of a bf16 pool."""
    pkg = _pkg()
    hkv, d, page = 8, 128, 256
    P = 2 ** 31 // (hkv * page * d) + 3
    k = torch.empty((P, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    small = Batch(28, hkv, 2, d, page, False, [300], [2], masks="chain")
    lse = torch.from_numpy(_lse(small)).cuda()
    a = small.dev()[0]
    want = torch.zeros(tuple(small.k.shape[:3]), device="cuda")
    pkg.attn_cache_weigh(a[0], lse, a[1], None, a[3], a[4], a[5], want, decay=0.0)
    k[P - 1], k[P - 2] = a[1][a[3][0, 0].long()], a[1][a[3][0, 1].long()]
    out = torch.zeros((P, hkv, page), device="cuda")
    pkg.attn_cache_weigh(a[0], lse, k, None, _i32([[P - 1, P - 2]]), a[4], a[5], out, decay=0.0)
    pkg.cache_check()
    assert torch.equal(out[P - 1], want[a[3][0, 0].long()])
    assert torch.equal(out[P - 2, :, :46], want[a[3][0, 1].long(), :, :46])


@pytest.mark.parametrize("hkv,G,d,page,B,ctx,T", [
    (16, 7, 128, 16, 28, (11, 22), (1, 401)),
    (16, 7, 64, 16, 28, (11, 22), (1, 401)),
    (8, 4, 128, 32, 100, (0, 700), (1, 80)),
    (8, 8, 128, 16, 150, (200, 1500), (1, 33)),
    (4, 16, 128, 64, 120, (0, 90), (0, 20)),
    (2, 100, 128, 16, 60, (0, 3000), (1, 2)),
])
def test_one_tile_and_several_in_turn(hkv, G, d, page, B, ctx, T):
    """e4m3 units whose codes go to the products as they are, next to ones that are widened: a role that sees only the
    keys of some units must not take one turn of a stage for another."""
    test_batches_against_torch(hkv, G, d, page, B, ctx, T, True)
