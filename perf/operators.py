"""The paged key/value cache and the attention that reads it: cases, inputs, plain forms and 64-bit values.

Three operators, as a decoding program calls them at every layer:

* write: the new tokens' K and V into a paged cache, copied (bf16) or quantised to e4m3 with one power-of-two scale
  for each (token, head);
* read:  cached positions back as packed bf16 K and V (what a packed prompt forward takes);
* tree:  attention of each sequence's drafted tokens over its cached context and, as the tree's mask allows, over each
  other; one drafted token per sequence is plain decoding.

Cache: k, v [num_pages, Hkv, page, d]; scale codes uint8 [num_pages, Hkv, page] with value = code * 2^(s - 127).
Position p of sequence b is row p % page of page block_table[b, p // page].
"""
import hashlib
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------------ cases

def _case(name, op, B, hq, hkv, d, page, cache, ctx, t, salt, tree=True):
    """ctx, t: (least, most) of the sequences' cached and new tokens; the lengths follow from the case alone."""
    return {"name": name, "op": op, "B": B, "hq": hq, "hkv": hkv, "d": d, "page": page, "cache": cache,
            "ctx_min": ctx[0], "ctx_max": ctx[1], "t_min": t[0], "t_max": t[1], "salt": salt, "tree": tree}


def listed():
    return [
        # one sequence decoding its next token: the append is pure latency
        _case("write one token bf16", "write", 1, 32, 8, 128, 16, "bf16", (701, 701), (1, 1), 1),
        # a decoding batch's step, quantised
        _case("write batch step e4m3", "write", 192, 32, 8, 128, 64, "e4m3", (0, 6000), (1, 1), 2),
        # ragged prompts going into the cache after their forward
        _case("write prompts e4m3", "write", 9, 32, 8, 128, 64, "e4m3", (0, 300), (900, 16384), 3),
        # a short prefix of a multi-head model with narrow heads, for a prompt over it
        _case("read prefixes bf16 d64", "read", 3, 16, 16, 64, 48, "bf16", (0, 0), (61, 517), 4),
        # long quantised prefixes read back for a packed prompt forward
        _case("read prefixes e4m3", "read", 6, 32, 8, 128, 128, "e4m3", (0, 0), (3000, 32768), 5),
        # one user, one token, a short context: latency
        _case("decode one sequence bf16", "tree", 1, 32, 8, 128, 16, "bf16", (517, 517), (1, 1), 6),
        # a decoding batch with ragged contexts, one token each
        _case("decode batch bf16", "tree", 48, 32, 8, 128, 64, "bf16", (900, 16384), (1, 1), 7),
        _case("decode batch e4m3", "tree", 64, 32, 8, 128, 64, "e4m3", (900, 16384), (1, 1), 8),
        # trees of drafted tokens over quantised contexts; some sequences draft nothing
        _case("draft trees e4m3", "tree", 24, 32, 8, 128, 32, "e4m3", (500, 8192), (0, 24), 9),
        # a multi-head model with 64-wide heads, chains of drafts
        _case("draft chains bf16 d64", "tree", 7, 32, 32, 64, 48, "bf16", (0, 5000), (2, 9), 10, tree=False),
        # one long document, the largest tree
        _case("draft tree long bf16", "tree", 1, 32, 8, 128, 128, "bf16", (131072, 131072), (64, 64), 11),
        # the same length quantised, one token of a wide group
        _case("decode long e4m3", "tree", 2, 64, 4, 128, 256, "e4m3", (100001, 262144), (1, 1), 12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "tree", "tree"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16, 32])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    cache = rng.choice(["bf16", "e4m3"])
    B = _log_int(rng, 1, 128)
    salt = rng.randrange(1 << 30)
    tokens = (2.4e8 if op == "tree" else 1.2e8) / (hkv * d)  # cached tokens in all: the bytes stay under the largest listed case's
    top = int(max(8, min(100000, tokens / B)))
    if op == "tree":
        t = rng.choice([(1, 1), (1, 1), (0, 5), (3, 17), (1, _log_int(rng, 2, 64))])
        top = int(max(8, min(top, 3.0e8 / (B * t[1] * hkv * group))))  # the plain form's scores fit too
        hi = _log_int(rng, 4, top)
        return _case("", op, B, hkv * group, hkv, d, page, cache, (rng.randrange(0, hi), hi), t, salt,
                     rng.random() < 0.7) | {"name": "drawn"}
    hi = _log_int(rng, 1, max(2, min(top, 40000)))
    ctx = (0, rng.choice([0, 1, 37, 1000])) if op == "write" else (0, rng.choice([0, 0, 5]))
    return _case("", op, B, hkv * group, hkv, d, page, cache, ctx, (rng.randrange(0, hi + 1), hi), salt) | {"name": "drawn"}


def _lengths(case):
    """Cached and new tokens of each sequence: the most once, the others spread over the logarithm."""
    h = hashlib.sha256(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()).digest()
    r = random.Random(int.from_bytes(h[:8], "big"))

    def some(lo, hi):
        v = [min(hi, max(lo, int(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 2)))) - 1)) for _ in range(case["B"])]
        v[r.randrange(case["B"])] = hi
        return v

    return some(case["ctx_min"], case["ctx_max"]), some(case["t_min"], case["t_max"])


# ------------------------------------------------------------------------------------------------ inputs

def _scale_codes(x):
    """e + 127 with e the least integer >= -126 for which max |x| of the last axis is at most 448 * 2^e."""
    m, e = torch.frexp(x.abs().amax(-1))  # |x| = m 2^e, m in [1/2, 1); 448 = 7/8 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return (torch.where(m > 0, e, torch.full_like(e, -126)).clamp_min(-126) + 127).to(torch.uint8)


def _two_to(s):
    """2^(s - 127) for codes s in [1, 254], exact."""
    return (s.to(torch.int32) << 23).view(torch.float32)


def _quantised(x):
    """x fp32 [..., d] -> e4m3 codes and scale codes."""
    s = _scale_codes(x)
    inv = ((254 - s.to(torch.int32)) << 23).view(torch.float32)  # 2^(127 - s)
    return (x * inv[..., None]).clamp(-448.0, 448.0).to(E4M3), s


def _values(shape, gen, dev):
    """Normal values, some channels several times larger, as keys and values have them."""
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)
    ch = torch.rand(shape[-1], generator=gen, device=dev)
    x *= torch.where(ch > 0.96, 4.0, 1.0) * (0.5 + ch)
    return x.to(torch.bfloat16)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    r = random.Random(int(seed))
    ctx, t = _lengths(case)
    B, hq, hkv, d, page = (case[k] for k in ("B", "hq", "hkv", "d", "page"))
    need = [-(-(c + n) // page) for c, n in zip(ctx, t)]
    wide = max(1, max(need)) + 1
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=dev, dtype=torch.int32)
    at = torch.cumsum(torch.tensor([0] + need), 0)
    row = at[:-1, None] + torch.arange(wide)[None, :]
    table = order[row.clamp_max(pages - 1).to(dev)]  # entries past a sequence's pages belong to others
    cu = torch.cumsum(torch.tensor([0] + t), 0)
    s = {"op": case["op"], "page": page, "d": d, "hq": hq, "hkv": hkv, "total": int(cu[-1]), "B": B,
         "longest": max(c + n for c, n in zip(ctx, t)), "max_new": max(t), "scale": 1.0 / math.sqrt(d),
         "table": table.contiguous(), "cu": cu.to(torch.int32).to(dev),
         "ctx": torch.tensor(ctx, dtype=torch.int32, device=dev), "ks": None, "vs": None}
    shape = (pages, hkv, page, d)
    if case["op"] == "write":
        # K and V as slices of the layer's joint projection
        joint = torch.empty((s["total"], (hq + 2 * hkv) * d), dtype=torch.bfloat16, device=dev)
        joint[:, hq * d:] = _values((s["total"], 2 * hkv, d), gen, dev).view(s["total"], -1)
        s["K"] = joint[:, hq * d:(hq + hkv) * d].view(-1, hkv, d)
        s["V"] = joint[:, (hq + hkv) * d:].view(-1, hkv, d)
        if case["cache"] == "e4m3":
            s["k"], s["v"] = (torch.zeros(shape, dtype=torch.uint8, device=dev).view(E4M3) for _ in range(2))
            s["ks"], s["vs"] = (torch.full(shape[:-1], 127, dtype=torch.uint8, device=dev) for _ in range(2))
        else:
            s["k"], s["v"] = (torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in range(2))
        return s
    for name in ("k", "v"):
        x = _values(shape, gen, dev)
        if case["cache"] == "e4m3":
            s[name], s[name + "s"] = _quantised(x.float())
        else:
            s[name] = x
    if case["op"] == "tree":
        s["Q"] = torch.randn((s["total"], hq, d), generator=gen, device=dev, dtype=torch.float32).to(torch.bfloat16)
        s["mask"] = None
        if case["tree"]:
            words = []
            for n in t:  # node i hangs on one of the nodes before it, or on the context
                seen = []
                for i in range(n):
                    up = r.randrange(-1, i) if i else -1
                    seen.append((1 << i) | (seen[up] if up >= 0 else 0))
                words += [w - (1 << 64) if w >> 63 else w for w in seen]
            s["mask"] = torch.tensor(words, dtype=torch.int64, device=dev)
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _places(s):
    """For every packed token: its page and its row there."""
    i = torch.arange(s["total"], device=s["cu"].device)
    b = torch.searchsorted(s["cu"], i, right=True) - 1
    pos = s["ctx"][b].long() + i - s["cu"][b].long()
    return s["table"][b, pos // s["page"]].long(), pos % s["page"]


def _plain_write(s):
    pg, off = _places(s)
    for x, cache, scale in ((s["K"], s["k"], s["ks"]), (s["V"], s["v"], s["vs"])):
        if scale is None:
            cache[pg, :, off] = x
        else:
            codes, sc = _quantised(x.float())
            cache.view(torch.uint8)[pg, :, off] = codes.view(torch.uint8)
            scale[pg, :, off] = sc
    return _cache_out(s)


def _cache_out(s):
    return {"k": s["k"], "v": s["v"]} if s["ks"] is None else {"k": s["k"], "v": s["v"], "ks": s["ks"], "vs": s["vs"]}


def _rows(cache, scale, pg, off):
    """fp32 rows [..., Hkv, d] of the cache at (page, row) places."""
    if scale is None:
        return cache[pg, :, off].float()
    return cache.view(torch.uint8)[pg, :, off].view(E4M3).float() * _two_to(scale[pg, :, off])[..., None]


def _plain_read(s):
    pg, off = _places(s)
    return [_rows(c, sc, pg, off).to(torch.bfloat16) for c, sc in ((s["k"], s["ks"]), (s["v"], s["vs"]))]


def _plain_tree(s):
    dev, B, G, L, T = s["Q"].device, s["B"], s["hq"] // s["hkv"], s["longest"], s["max_new"]
    ctx, cu = s["ctx"].long(), s["cu"].long()
    n = cu[1:] - cu[:-1]
    j = torch.arange(L, device=dev)
    pos = torch.minimum(j[None], (ctx + n - 1).clamp_min(0)[:, None])
    pg, off = torch.gather(s["table"].long(), 1, pos // s["page"]), pos % s["page"]
    i = torch.arange(T, device=dev)
    tok = (cu[:-1, None] + i[None]).clamp_max(s["total"] - 1)  # [B, T]
    q = s["Q"].float()[tok].view(B, T, s["hkv"], G, s["d"])
    u = j[None] - ctx[:, None]  # drafted node of key j, negative in the context
    words = s["mask"][tok] if s["mask"] is not None else (torch.full_like(i, 2) << i)[None].expand(B, T) - 1
    bit = (words[:, :, None] >> u.clamp(0, 63)[:, None, :]) & 1
    sees = ((u < 0)[:, None, :] | ((u < n[:, None])[:, None, :] & (bit == 1))) & (i[None] < n[:, None])[:, :, None]
    x = torch.einsum("bthgd,blhd->bthgl", q, _rows(s["k"], s["ks"], pg, off)) * s["scale"]
    x = x.masked_fill(~sees[:, :, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    o = torch.einsum("bthgl,blhd->bthgd", p, _rows(s["v"], s["vs"], pg, off)) / torch.where(l > 0, l, torch.ones_like(l))
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf))[..., 0]
    k = torch.arange(s["total"], device=dev)
    b = torch.searchsorted(cu, k, right=True) - 1
    at = k - cu[b]
    return {"O": o[b, at].reshape(s["total"], s["hq"], s["d"]).to(torch.bfloat16),
            "LSE": lse[b, at].reshape(s["total"], s["hq"]).t().contiguous()}


def run(s):
    if own:
        import online_softmax_flashattention_attention_gb300 as attn
        if s["op"] == "write":
            attn.attn_cache_write(s["K"], s["V"], s["k"], s["v"], s["table"], s["cu"], start_lens=s["ctx"],
                                  k_scale=s["ks"], v_scale=s["vs"])
            return _cache_out(s)
        if s["op"] == "read":
            K, V = attn.attn_cache_read(s["k"], s["v"], s["table"], s["cu"], s["total"], start_lens=s["ctx"],
                                        k_scale=s["ks"], v_scale=s["vs"])
            return [K, V]
        O, LSE = attn.attn_fwd_tree(s["Q"], s["k"], s["v"], s["table"], s["ctx"], s["cu"], s["max_new"],
                                    tree_mask=s["mask"], k_scale=s["ks"], v_scale=s["vs"], scale=s["scale"])
        return {"O": O, "LSE": LSE}
    return {"write": _plain_write, "read": _plain_read, "tree": _plain_tree}[s["op"]](s)


# ------------------------------------------------------------------------------------------------ work

def work(case):
    ctx, t = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    row = 2 * hkv * (2 * d if case["cache"] == "bf16" else d + 1)  # one cached token, K and V
    n = sum(t)
    if case["op"] != "tree":
        return {"bytes": n * (row + 2 * hkv * 2 * d), "flops": 0 if case["cache"] == "bf16" else 2 * n * hkv * d * 2}
    keys = sum(c + k for c, k in zip(ctx, t) if k > 0)
    return {"bytes": keys * row + n * hq * (4 * d + 4) + (8 * n if case["tree"] else 0),
            "flops": 4 * d * hq * sum(k * (c + k) for c, k in zip(ctx, t))}


# ------------------------------------------------------------------------------------------------ 64 bits

def _power(e):
    """2^e in 64 bits from its bits: a power function on the device may miss it by an ulp, which turns ties."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _on_grid(y):
    """y to the nearest e4m3 value, ties to even, by arithmetic in 64 bits (|y| <= 448)."""
    _, e = torch.frexp(y)
    step = _power((e - 1).clamp_min(-6) - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    """Sequence by sequence and position by position from the definitions, in 64 bits."""
    s = prepare(case, seed)
    ctx, t = _lengths(case)
    page, d, hkv, G = case["page"], case["d"], case["hkv"], case["hq"] // case["hkv"]
    table = s["table"].cpu()
    f8 = case["cache"] == "e4m3"

    def slots(b, first, count):
        """(page, row) of the positions first .. first + count - 1 of sequence b."""
        p = torch.arange(first, first + count)
        return table[b][p // page].long().to("cuda"), (p % page).to("cuda")

    def cached(name, b, first, count):
        pg, off = slots(b, first, count)
        flat = pg * page * hkv + off  # row of head 0; head h is page rows further
        flat = flat[:, None] + torch.arange(hkv, device="cuda")[None] * page
        x = s[name].view(torch.uint8).view(-1, d * (1 if f8 else 2))[flat].view(E4M3 if f8 else torch.bfloat16).double()
        if f8:
            x = x * _power(s[name + "s"].view(-1)[flat].to(torch.int64) - 127)[..., None]
        return x  # [count, hkv, d]

    first = 0
    if case["op"] == "write":
        out = {k: v.double() if k in ("k", "v") else v.clone() for k, v in _cache_out(s).items()}
        for b in range(case["B"]):
            if not t[b]:
                continue
            pg, off = slots(b, ctx[b], t[b])
            for src, name in (("K", "k"), ("V", "v")):
                x = s[src][first:first + t[b]].double()
                if f8:
                    top = x.abs().amax(-1)
                    e = torch.log2((top / 448.0).clamp_min(2.0 ** -130)).round().to(torch.int64) - 1
                    for _ in range(2):  # the least e with top <= 448 * 2^e, by that comparison
                        e += (top > 448.0 * _power(e)).to(torch.int64)
                    e = e.clamp_min(-126)
                    out[name + "s"][pg, :, off] = (e + 127).to(torch.uint8)
                    x = _on_grid(x * _power(-e)[..., None])
                out[name][pg, :, off] = x
            first += t[b]
        return out
    if case["op"] == "read":
        return [torch.cat([cached(name, b, ctx[b], t[b]) for b in range(case["B"])]) for name in ("k", "v")]
    outs, lses = [], []
    for b in range(case["B"]):
        if not t[b]:
            continue
        K, V = (cached(name, b, 0, ctx[b] + t[b]).transpose(0, 1) for name in ("k", "v"))  # [hkv, L, d]
        sees = torch.ones(t[b], ctx[b] + t[b], dtype=torch.bool)
        words = None if s["mask"] is None else s["mask"][first:first + t[b]].tolist()
        for i in range(t[b]):
            for u in range(t[b]):
                sees[i, ctx[b] + u] = u <= i if words is None else bool((words[i] >> u) & 1)
        sees = sees.repeat_interleave(G, 0).to("cuda")
        q = s["Q"][first:first + t[b]].double().view(t[b], hkv, G, d).transpose(0, 1).reshape(hkv, t[b] * G, d)
        o, e = [], []
        for h in range(hkv):
            z = (q[h] @ K[h].t()) / math.sqrt(d)
            z = torch.where(sees, z, torch.full_like(z, -math.inf))
            e.append(torch.logsumexp(z, -1))
            w = torch.exp(z - e[-1][:, None])
            o.append(torch.where(sees.any(-1)[:, None], w @ V[h], torch.zeros_like(q[h])))
        outs.append(torch.stack(o).view(hkv, t[b], G, d).transpose(0, 1).reshape(t[b], hkv * G, d))
        lses.append(torch.stack(e).view(hkv, t[b], G).transpose(1, 2).reshape(hkv * G, t[b]))
        first += t[b]
    if not outs:
        return {"O": s["Q"].double(), "LSE": torch.zeros((case["hq"], 0), dtype=torch.float64)}
    return {"O": torch.cat(outs), "LSE": torch.cat(lses, 1)}
