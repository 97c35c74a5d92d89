"""The operators as a serving program chains them: rotate, prompt attention, cache write, weigh, evict, then
decoding steps over the smaller cache, held against 64-bit attention over exactly the tokens kept."""
import math

import numpy as np
import pytest
import torch

from cache_ref import HALF_BF16

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d,interleaved", [(64, True), (128, False)])
def test_prompts_then_bounded_decoding(d, interleaved, f8):
    import online_softmax_flashattention_attention_gb300 as attn
    g = torch.Generator(device="cuda")
    g.manual_seed(41)
    hkv, G, page, keep, lens = 2, 4, 16, 100, [260, 40, 101]
    hq, B, total, scale = hkv * G, 3, sum(lens), 1 / math.sqrt(d)
    freq = (10000.0 ** (-torch.arange(d // 2, device="cuda") / (d // 2))).float()
    qw, kw = (1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    cu = _i32([0] + np.cumsum(lens).tolist())
    pages = [-(-(n + 8) // page) for n in lens]
    table = torch.zeros((B, max(pages)), dtype=torch.int32, device="cuda")
    order = torch.randperm(sum(pages), generator=g, device="cuda").to(torch.int32)
    for b in range(B):
        table[b, :pages[b]] = order[sum(pages[:b]):sum(pages[:b + 1])]
    shape = (sum(pages), hkv, page, d)
    sc = {}
    if f8:
        k, v = (torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
        sc = {n: torch.ones(shape[:3], dtype=torch.uint8, device="cuda") for n in ("k_scale", "v_scale")}
    else:
        k, v = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    weights = torch.full(shape[:3], float("nan"), device="cuda")  # fresh tokens start from 0 whatever it holds

    def project(n):
        return torch.randn((n, hq + 2 * hkv, d), generator=g, device="cuda").to(torch.bfloat16)

    joint = project(total)
    Q, K = attn.attn_qk_rotate(joint[:, :hq], joint[:, hq:hq + hkv], cu, freq, q_weight=qw, k_weight=kw, interleaved=interleaved)
    V = joint[:, hq + hkv:]
    O, LSE = attn.attn_fwd_prompt(Q, K, V, cu, cu, max(lens))
    attn.attn_cache_write(K, V, k, v, table, cu, **sc)
    K, V = attn.attn_cache_read(k, v, table, cu, total, **sc)  # what the cache holds, for the reference
    if f8:  # the weights are those of the cached keys
        O, LSE = attn.attn_fwd_prompt(Q, K, V, cu, cu, max(lens))
    ks = {"k_scale": sc["k_scale"]} if f8 else {}
    attn.attn_cache_weigh(Q, LSE, k, weights, table, None, cu, **ks)
    # every row's weights sum to 1: all together to the number of rows of a head's group
    for b, n in enumerate(lens):
        w = weights[table[b].long()].transpose(0, 1).reshape(hkv, -1)[:, :n].double().sum(-1)
        assert bool(((w - G * n).abs() <= 2.0 ** -16 * G * n).all())
    kept, now = attn.attn_cache_evict(k, v, weights, table, _i32(lens), keep, sink=4, recent=20, **sc)
    attn.cache_check()
    assert now.tolist() == [min(n, keep) for n in lens]
    assert kept[1, 0, 40:].eq(-1).all()
    alive = [[(K[sum(lens[:b]):][kept[b, h, :int(now[b])].long(), h], V[sum(lens[:b]):][kept[b, h, :int(now[b])].long(), h])
              for h in range(hkv)] for b in range(B)]
    for step in range(3):
        joint = project(B)
        one = _i32(range(B + 1))
        at = _i32([n + step for n in lens])  # positions of the text, not places in the cache
        q, kk = attn.attn_qk_rotate(joint[:, :hq], joint[:, hq:hq + hkv], one, freq, positions=at, q_weight=qw, k_weight=kw,
                                    interleaved=interleaved)
        vv = joint[:, hq + hkv:]
        attn.attn_cache_write(kk, vv, k, v, table, one, start_lens=now, **sc)
        kk, vv = attn.attn_cache_read(k, v, table, one, B, start_lens=now, **sc)
        O, LSE = attn.attn_fwd_tree(q, k, v, table, now, one, 1, **sc)
        attn.attn_cache_weigh(q, LSE, k, weights, table, now, one, **ks)
        attn.cache_check()
        for b in range(B):
            for h in range(hkv):
                alive[b][h] = tuple(torch.cat((x, y[b:b + 1, h])) for x, y in zip(alive[b][h], (kk, vv)))
                kr, vr = (x.double() for x in alive[b][h])
                z = q[b, h * G:(h + 1) * G].double() @ kr.t() * scale
                p = torch.softmax(z, -1)
                want, size = p @ vr, p @ vr.abs()
                # O's rounding, the probabilities' (2^-8 each), and 2^-10 for the e4m3 form of q and all in fp32
                assert bool(((O[b, h * G:(h + 1) * G].double() - want).abs() <= HALF_BF16 * want.abs() + (HALF_BF16 + 2.0 ** -10) * size).all())
        now = now + 1
    for b in range(B):  # a step adds G to a head's weights in all
        w = weights[table[b].long()].transpose(0, 1).reshape(hkv, -1)[:, :int(now[b])]
        assert bool(torch.isfinite(w).all())
