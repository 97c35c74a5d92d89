"""Weights through a serving run: what a prompt's keys received, moved by eviction, and added to by decoding
steps over the smaller cache, held against the definition position by position and in all."""
import math

import numpy as np
import pytest
import torch

from cache_ref import U
from prompt_ref import f64, ref_weigh

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_steps_add_to_the_weights_that_eviction_moved(d, f8, other):
    """A row's weights are probabilities, so that a step adds G to a head's weights in all.  Off by: what
    ref_weigh allows every weight, and for the sum to be G what the LSE may be off by, as cache_ref says:
    ds = (d + 2) U B (scores at most B), for e4m3 the same loss of the query that the weights have, and the
    sum's (n / 16 + 64) U, a logarithm and its product."""
    import online_softmax_flashattention_attention_gb300 as attn
    g = torch.Generator(device="cuda")
    g.manual_seed(43)
    hkv, G, page, keep, lens = 2, 4, 16, 100, [260, 40, 101]
    hq, B, total, scale = hkv * G, 3, sum(lens), 1 / math.sqrt(d)
    cu = _i32([0] + np.cumsum(lens).tolist())
    width = -(-(max(lens) + 8) // page)
    order = torch.randperm(2 * B * width, generator=g, device="cuda").to(torch.int32).view(2, B, width)
    table, to = order[0].contiguous(), order[1].contiguous()
    shape = (2 * B * width, hkv, page, d)
    sc, ks = {}, {}
    if f8:
        k, v = (torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
        sc = {n: torch.ones(shape[:3], dtype=torch.uint8, device="cuda") for n in ("k_scale", "v_scale")}
        ks = {"k_scale": sc["k_scale"]}
    else:
        k, v = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    weights = torch.full(shape[:3], float("nan"), device="cuda")

    def rows(n, heads):
        return torch.randn((n, heads, d), generator=g, device="cuda").to(torch.bfloat16)

    Q = rows(total, hq)
    attn.attn_cache_write(rows(total, hkv), rows(total, hkv), k, v, table, cu, **sc)
    K, V = attn.attn_cache_read(k, v, table, cu, total, **sc)
    O, LSE = attn.attn_fwd_prompt(Q, K, V, cu, cu, max(lens))
    attn.attn_cache_weigh(Q, LSE, k, weights, table, None, cu, decay=0.0, **ks)
    kept, now = attn.attn_cache_evict(k, v, weights, table, _i32(lens), keep, sink=4, recent=20, out_table=to if other else None, **sc)
    attn.cache_check()
    assert now.tolist() == [min(n, keep) for n in lens]
    at = to if other else table
    one, host = _i32(range(B + 1)), at.cpu().numpy()

    def all_of(n):
        w = weights[at.long()].transpose(1, 2).reshape(B, hkv, -1).double()
        return torch.stack([w[b, :, :int(n[b])].sum(-1) for b in range(B)]).cpu().numpy()

    for step in range(3):
        q = rows(B, hq)
        attn.attn_cache_write(rows(B, hkv), rows(B, hkv), k, v, at, one, start_lens=now, **sc)
        O, LSE = attn.attn_fwd_tree(q, k, v, at, now, one, 1, **sc)
        before, sums = weights.cpu().numpy(), all_of(now)
        attn.attn_cache_weigh(q, LSE, k, weights, at, now, one, **ks)
        attn.cache_check()
        want, tol = ref_weigh(f64(q), f64(LSE), f64(k), sc["k_scale"].cpu().numpy() if f8 else None, host, now.tolist(),
                              list(range(B + 1)), page, scale, 1.0, before.astype(np.float64), before.astype(np.float64))
        got = f64(weights)
        assert np.array_equal(np.isnan(got), np.isnan(want))  # (places of no sequence)
        ok = ~np.isnan(want)
        assert np.all(np.abs(got[ok] - want[ok]) <= tol[ok])
        grown = all_of(now + 1) - sums
        for b in range(B):
            n = int(now[b]) + 1
            pg, row = host[b, np.arange(n) // page], np.arange(n) % page
            for h in range(hkv):
                kh = f64(k)[pg, h, row] * (1.0 if not f8 else np.exp2(sc["k_scale"].cpu().numpy()[pg, h, row] - 127.0)[:, None])
                qh = f64(q)[b, h * G:(h + 1) * G]
                # (e4m3: a query value in either form is off by at most 2^-17 of its row's largest's power of two)
                big = scale * (np.abs(qh) @ np.abs(kh).T).max()
                lost = scale * 2.0 ** -17 * (np.abs(qh).max() * np.abs(kh).sum(1)).max() if f8 else 0.0
                top = np.abs(f64(LSE)[h * G:(h + 1) * G, b]).max()
                lse = (d + 2) * U * big + lost + (n / 16 + 64) * U + 8 * U * (1 + top)
                assert abs(grown[b, h] - G) <= tol[pg, h, row].sum() + 1.01 * G * lse
        now = now + 1
