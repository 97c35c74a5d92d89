"""Prompts with grouped heads and a cache of bounded length: cases, inputs, plain forms and 64-bit values.

Four operators, as a serving program calls them at every layer:

* rotate: the norm of every query and key head and the rotation by position, from the joint projection;
* prompt: causal attention of packed prompts whose query heads share K/V heads, some of them over a prefix;
* weigh:  the attention weight that every cached key received from a call's queries, added to what it had;
* evict:  each sequence's keys of least accumulated weight dropped, the others packed into new pages.

Cache: k, v [num_pages, Hkv, page, d], weights fp32 [num_pages, Hkv, page]; an e4m3 cache has scale codes uint8
[num_pages, Hkv, page] with value = code * 2^(s - 127).  Position p of sequence b is row p % page of page
block_table[b, p // page].
"""
import hashlib
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ cases

def _case(name, op, B, hq, hkv, d, ctx, t, salt, **more):
    """ctx, t: (least, most) of the sequences' tokens before the call and in it; the lengths follow from the case."""
    return {"name": name, "op": op, "B": B, "hq": hq, "hkv": hkv, "d": d, "ctx_min": ctx[0], "ctx_max": ctx[1],
            "t_min": t[0], "t_max": t[1], "salt": salt} | more


def _rotate(name, B, hq, hkv, d, ctx, t, salt, rot, norm, pairs):
    return _case(name, "rotate", B, hq, hkv, d, ctx, t, salt, rot=rot, norm=norm, interleaved=pairs)


def _prompt(name, B, hq, hkv, d, ctx, t, salt):
    return _case(name, "prompt", B, hq, hkv, d, ctx, t, salt)


def _weigh(name, B, hq, hkv, d, page, cache, ctx, t, salt, decay):
    return _case(name, "weigh", B, hq, hkv, d, ctx, t, salt, page=page, cache=cache, decay=decay)


def _evict(name, B, hkv, d, page, cache, t, salt, keep, sink, recent):
    return _case(name, "evict", B, hkv, hkv, d, (0, 0), t, salt, page=page, cache=cache, keep=keep, sink=sink, recent=recent)


def listed():
    return [
        # one sequence's next token, far into its context: latency
        _rotate("rotate one token", 1, 32, 8, 128, (100000, 100000), (1, 1), 1, 128, True, False),
        # a decoding batch of narrow heads without norms, a quarter of each rotated in neighbouring pairs
        _rotate("rotate batch step d64", 61, 32, 8, 64, (0, 6000), (1, 3), 2, 16, False, True),
        # ragged prompts after their projection
        _rotate("rotate prompts", 9, 32, 8, 128, (0, 300), (900, 16384), 3, 128, True, False),
        # one short question: latency
        _prompt("prompt short", 1, 32, 8, 128, (0, 0), (77, 77), 4),
        # further turns of conversations over their prefixes, narrow heads
        _prompt("prompts over prefixes d64", 7, 16, 4, 64, (0, 5000), (61, 517), 5),
        # a batch of ragged prompts
        _prompt("prompts ragged", 9, 32, 8, 128, (0, 0), (900, 8192), 6),
        # one long document
        _prompt("prompt long", 1, 32, 8, 128, (0, 0), (16384, 16384), 7),
        # one sequence's next token over a short context: latency
        _weigh("weigh one token bf16", 1, 32, 8, 128, 16, "bf16", (517, 517), (1, 1), 8, 1.0),
        # a decoding batch with ragged contexts, quantised, old weights fading
        _weigh("weigh batch e4m3", 64, 32, 8, 128, 64, "e4m3", (900, 16384), (1, 1), 9, 0.98),
        # every query of a prompt counts
        _weigh("weigh prompt bf16", 1, 32, 8, 128, 64, "bf16", (0, 0), (8192, 8192), 10, 0.0),
        # one conversation back to its budget: latency
        _evict("evict one sequence bf16", 1, 8, 128, 16, "bf16", (1733, 1733), 11, 1024, 4, 64),
        # a batch of prompts cut to their budgets, some shorter than it
        _evict("evict batch e4m3", 48, 8, 128, 64, "e4m3", (900, 16384), 12, 4096, 16, 256),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "prompt", "prompt", "weigh", "weigh", "evict"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    hq = hkv * group
    page = rng.choice([16, 32, 48, 64, 128, 256])
    cache = rng.choice(["bf16", "e4m3"])
    B = _log_int(rng, 1, 64)
    salt = rng.randrange(1 << 30)
    if op == "rotate":
        hi = _log_int(rng, 1, max(2, int(min(16384, 2.0e8 / (B * (hq + hkv) * d)))))
        rot = rng.choice([r for r in (0, 16, 32, 64, 96, 128) if r <= d])
        return _rotate("drawn", B, hq, hkv, d, (0, rng.choice([0, 37, 5000, 1 << 20])), (rng.randrange(0, hi + 1), hi), salt,
                       rot, rng.random() < 0.6, rng.random() < 0.4)
    if op == "prompt":
        # the longest sequences' scores stay under the longest listed case's
        n = int(min(16384, math.sqrt(6.0e11 / (B * hq * d))))
        hi = _log_int(rng, 1, max(2, n))
        before = rng.choice([0, 0, max(0, n - hi)])
        return _prompt("drawn", B, hq, hkv, d, (0, before), (rng.randrange(0, hi + 1), hi), salt)
    if op == "weigh":
        n = int(max(8, min(40000, 2.4e8 / (B * hkv * d))))
        t = rng.choice([(1, 1), (1, 1), (0, 5), (1, _log_int(rng, 2, 64)), (1, _log_int(rng, 64, 2048))])
        hi = _log_int(rng, 4, int(max(8, min(n, 1.2e11 / (B * t[1] * hq * d)))))
        return _weigh("drawn", B, hq, hkv, d, page, cache, (rng.randrange(0, hi), hi), t, salt, rng.choice([0.0, 0.9, 1.0]))
    n = _log_int(rng, 2, int(max(8, min(100000, 2.0e8 / (B * hkv * d)))))
    keep = _log_int(rng, 1, n)
    sink = rng.choice([0, 0, min(4, keep)])
    return _evict("drawn", B, hkv, d, page, cache, (rng.randrange(0, n + 1), n), salt, keep, sink,
                  rng.choice([0, (keep - sink) // 3, keep - sink]))


def _lengths(case):
    """Tokens before the call and in it of each sequence: the most once, the others spread over the logarithm."""
    h = hashlib.sha256(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()).digest()
    r = random.Random(int.from_bytes(h[:8], "big"))

    def some(lo, hi):
        v = [min(hi, max(lo, int(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 2)))) - 1)) for _ in range(case["B"])]
        v[r.randrange(case["B"])] = hi
        return v

    return some(case["ctx_min"], case["ctx_max"]), some(case["t_min"], case["t_max"])


# ------------------------------------------------------------------------------------------------ inputs

def _values(shape, gen):
    """Normal values, some channels several times larger, as keys and values have them."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    ch = torch.rand(shape[-1], generator=gen, device="cuda")
    x *= torch.where(ch > 0.96, 4.0, 1.0) * (0.5 + ch)
    return x.to(torch.bfloat16)


def _quantised(x):
    """fp32 rows -> e4m3 codes and scale codes s = e + 127, e the least with max |x| <= 448 * 2^e."""
    m, e = torch.frexp(x.abs().amax(-1))  # |x| = m 2^e, m in [1/2, 1); 448 = 7/8 * 2^9
    s = (torch.where(m <= 0.875, e - 9, e - 8) + 127).to(torch.uint8)
    inv = ((254 - s.to(torch.int32)) << 23).view(torch.float32)
    return (x * inv[..., None]).clamp(-448.0, 448.0).to(E4M3), s


def _i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _offsets(lengths):
    return torch.cumsum(torch.tensor([0] + list(lengths)), 0)


def _pages(lengths, page, gen, spare):
    """Block table of sequences of these lengths over a shuffled pool with `spare` pages nobody has."""
    need = [-(-n // page) for n in lengths]
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int32)
    row = _offsets(need)[:-1, None] + torch.arange(max(1, max(need)))[None, :]
    return order[row.clamp_max(total - 1).cuda()].contiguous(), order, sum(need)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    ctx, t = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    cu = _offsets(t)
    s = {"op": case["op"], "d": d, "hq": hq, "hkv": hkv, "B": case["B"], "ctx_host": ctx, "t_host": t,
         "cu": cu.to(torch.int32).cuda(), "ctx": _i32(ctx), "total": int(cu[-1]), "scale": 1.0 / math.sqrt(d)}
    if case["op"] == "rotate":
        # queries and keys as slices of the layer's joint projection
        joint = _values((s["total"], hq + 2 * hkv, d), gen)
        s["Q"], s["K"] = joint[:, :hq], joint[:, hq:hq + hkv]
        s["qw"], s["kw"] = (((1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16) for _ in range(2))
                            if case["norm"] else (None, None))
        r = case["rot"]
        s["freq"] = None if r == 0 else (500000.0 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)).float()
        s["interleaved"] = case["interleaved"]
        return s
    if case["op"] == "prompt":
        n = [c + k for c, k in zip(ctx, t)]
        cu_k = _offsets(n)
        s["cu_k"], s["max_q"] = cu_k.to(torch.int32).cuda(), max(t)
        if max(ctx) == 0:
            joint = _values((s["total"], hq + 2 * hkv, d), gen)
            s["Q"], s["K"], s["V"] = joint[:, :hq], joint[:, hq:hq + hkv], joint[:, hq + hkv:]
        else:  # the prefixes' rows, read back from a cache, with the new ones behind them
            s["Q"] = _values((s["total"], hq, d), gen)
            s["K"], s["V"] = (_values((int(cu_k[-1]), hkv, d), gen) for _ in range(2))
        return s
    page = s["page"] = case["page"]
    n = [c + k for c, k in zip(ctx, t)]
    s["table"], order, used = _pages(n, page, gen, 3 + case["B"] * -(-case.get("keep", 0) // page))
    s["ks"] = s["vs"] = None
    shape = (order.numel(), hkv, page, d)
    for name in ("k", "v") if case["op"] == "evict" else ("k",):
        s[name] = _values(shape, gen)
        if case["cache"] == "e4m3":
            s[name], s[name + "s"] = _quantised(s[name].float())
    # weights as prompts leave them: a few keys have most
    s["w"] = torch.exp(2.0 * torch.randn(shape[:3], generator=gen, device="cuda") - 3.0)
    if case["op"] == "evict":
        s["keep"], s["sink"], s["recent"] = case["keep"], case["sink"], case["recent"]
        s["n"] = s["ctx"] + _i32(t)
        wide = -(-case["keep"] // page)
        s["to"] = order[used + torch.arange(case["B"] * wide, device="cuda")].view(case["B"], wide).contiguous()
        return s
    s["decay"], s["out"] = case["decay"], torch.zeros_like(s["w"])
    s["Q"] = torch.randn((s["total"], hq, d), generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    s["LSE"] = torch.empty((hq, s["total"]), dtype=torch.float32, device="cuda")
    for b in range(case["B"]):  # what the attention of these queries returned
        if t[b]:
            z = torch.logsumexp(_seen_scores(s, b), -1).view(hkv, t[b], -1)
            s["LSE"][:, int(cu[b]):int(cu[b + 1])] = z.transpose(1, 2).reshape(hq, t[b])
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _two_to(s):
    """2^(s - 127) for codes s in [1, 254], exact."""
    return (s.to(torch.int32) << 23).view(torch.float32)


def _slots(s, table, b, pos):
    return table[b].long()[pos // s["page"]], pos % s["page"]


def _keys(s, b, n):
    """fp32 keys [hkv, n, d] of a sequence."""
    pg, row = _slots(s, s["table"], b, torch.arange(n, device="cuda"))
    if s["ks"] is None:
        return s["k"][pg, :, row].float().transpose(0, 1)
    codes = s["k"].view(torch.uint8)[pg, :, row].view(E4M3)
    return (codes.float() * _two_to(s["ks"][pg, :, row])[..., None]).transpose(0, 1)


def _seen_scores(s, b):
    """Scores [hkv, T * G, n] of a sequence's rows (token, head of the group), -inf where a row does not look."""
    c, t, G = s["ctx_host"][b], s["t_host"][b], s["hq"] // s["hkv"]
    first = sum(s["t_host"][:b])
    q = s["Q"][first:first + t].float().view(t, -1, G, s["d"]).transpose(0, 1).reshape(-1, t * G, s["d"])
    z = (q @ _keys(s, b, c + t).transpose(1, 2)) * s["scale"]
    sees = torch.arange(c + t, device="cuda")[None, :] <= c + torch.arange(t, device="cuda").repeat_interleave(G)[:, None]
    return z.masked_fill_(~sees, -math.inf)


def _plain_rotate(s):
    i = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(s["cu"], i, right=True) - 1
    pos = s["ctx"][b].long() + i - s["cu"][b].long()
    out = []
    for x, w in ((s["Q"], s["qw"]), (s["K"], s["kw"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        if s["freq"] is not None:
            r = 2 * s["freq"].numel()
            angle = pos.double()[:, None] * s["freq"].double()
            cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
            first, second = ((x[..., 0:r:2], x[..., 1:r:2]) if s["interleaved"] else (x[..., :r // 2], x[..., r // 2:r]))
            turned = (first * cos - second * sin, second * cos + first * sin)
            turned = torch.stack(turned, -1).flatten(-2) if s["interleaved"] else torch.cat(turned, -1)
            x = torch.cat((turned, x[..., r:]), -1)
        out.append(x.to(torch.bfloat16))
    return out


def _plain_prompt(s):
    G, d = s["hq"] // s["hkv"], s["d"]
    O = torch.empty((s["total"], s["hq"], d), dtype=torch.bfloat16, device="cuda")
    LSE = torch.empty((s["hq"], s["total"]), dtype=torch.float32, device="cuda")
    q0 = k0 = 0
    for c, t in zip(s["ctx_host"], s["t_host"]):
        K, V = s["K"][k0:k0 + c + t].float(), s["V"][k0:k0 + c + t].float()
        ahead = torch.arange(c + t, device="cuda")[None, :] > c + torch.arange(t, device="cuda")[:, None]
        for h in range(s["hq"] if t else 0):
            z = (s["Q"][q0:q0 + t, h].float() @ K[:, h // G].t()) * s["scale"]
            z.masked_fill_(ahead, -math.inf)
            m = z.amax(-1, keepdim=True)
            p = torch.exp(z - m)
            l = p.sum(-1, keepdim=True)
            O[q0:q0 + t, h] = ((p @ V[:, h // G]) / l).to(torch.bfloat16)
            LSE[h, q0:q0 + t] = (m + torch.log(l))[:, 0]
        q0, k0 = q0 + t, k0 + c + t
    return {"O": O, "LSE": LSE}


def _plain_weigh(s):
    hkv, first = s["hkv"], 0
    for b, (c, t) in enumerate(zip(s["ctx_host"], s["t_host"])):
        if t:
            pg, row = _slots(s, s["table"], b, torch.arange(c + t, device="cuda"))
            lse = s["LSE"][:, first:first + t].view(hkv, -1, t).transpose(1, 2).reshape(hkv, -1, 1)
            got = torch.exp(_seen_scores(s, b) - lse).sum(1).t()
            if s["decay"] != 0.0:
                got[:c] += s["decay"] * s["w"][pg[:c], :, row[:c]]
            s["out"][pg, :, row] = got
        first += t
    return s["out"]


def _pools(s):
    return [x for x in (s["k"], s["v"], s["ks"], s["vs"], s["w"]) if x is not None]


def _plain_evict(s):
    keep, sink, recent, hkv = s["keep"], s["sink"], s["recent"], s["hkv"]
    kept = torch.full((s["B"], hkv, keep), -1, dtype=torch.int32, device="cuda")
    heads = torch.arange(hkv, device="cuda")[:, None]
    for b, n in enumerate(s["t_host"]):
        pos = torch.arange(n, device="cuda").expand(hkv, n)
        if n > keep:
            pg, row = _slots(s, s["table"], b, torch.arange(sink, n - recent, device="cuda"))
            order = torch.sort(s["w"][pg, :, row].t(), dim=-1, descending=True, stable=True).indices
            best = sink + order[:, :keep - sink - recent]
            pos = torch.cat((pos[:, :sink], torch.sort(best, -1).values, pos[:, n - recent:]), -1)
        m = pos.shape[1]
        kept[b, :, :m] = pos.to(torch.int32)
        pg, row = _slots(s, s["table"], b, pos)
        to_pg, to_row = _slots(s, s["to"], b, torch.arange(m, device="cuda"))
        for x in _pools(s):
            x = x.view(torch.uint8) if x.dtype == E4M3 else x
            x[to_pg, heads, to_row] = x[pg, heads, row]
    return _evict_out(s, kept, torch.clamp(s["n"], max=keep))


def _evict_out(s, kept, lens):
    return {"kept": kept, "lens": lens} | {k: s[k] for k in ("k", "v", "ks", "vs", "w") if s[k] is not None}


def run(s):
    if not own:
        return {"rotate": _plain_rotate, "prompt": _plain_prompt, "weigh": _plain_weigh, "evict": _plain_evict}[s["op"]](s)
    import online_softmax_flashattention_attention_gb300 as attn
    if s["op"] == "rotate":
        Q, K = attn.attn_qk_rotate(s["Q"], s["K"], s["cu"], s["freq"], start_lens=s["ctx"], q_weight=s["qw"],
                                   k_weight=s["kw"], eps=EPS, interleaved=s["interleaved"])
        return [Q, K]
    if s["op"] == "prompt":
        O, LSE = attn.attn_fwd_prompt(s["Q"], s["K"], s["V"], s["cu"], s["cu_k"], s["max_q"], scale=s["scale"])
        return {"O": O, "LSE": LSE}
    if s["op"] == "weigh":
        return attn.attn_cache_weigh(s["Q"], s["LSE"], s["k"], s["w"], s["table"], s["ctx"], s["cu"], out=s["out"],
                                     decay=s["decay"], k_scale=s["ks"], scale=s["scale"])
    kept, lens = attn.attn_cache_evict(s["k"], s["v"], s["w"], s["table"], s["n"], s["keep"], sink=s["sink"],
                                       recent=s["recent"], out_table=s["to"], k_scale=s["ks"], v_scale=s["vs"])
    return _evict_out(s, kept, lens)


# ------------------------------------------------------------------------------------------------ work

def work(case):
    ctx, t = _lengths(case)
    op, hq, hkv, d = case["op"], case["hq"], case["hkv"], case["d"]
    total = sum(t)
    pairs = sum(k * c + k * (k + 1) // 2 for c, k in zip(ctx, t))  # visible (token, key) pairs
    if op == "rotate":
        values = total * (hq + hkv) * d
        return {"bytes": 4 * values, "flops": values * (4 if case["norm"] else 0) + 3 * total * (hq + hkv) * case["rot"]}
    keys = sum(c + k for c, k in zip(ctx, t) if k > 0)
    if op == "prompt":
        return {"bytes": total * hq * (4 * d + 4) + keys * hkv * 4 * d, "flops": 4 * d * hq * pairs}
    row = 2 * d if case["cache"] == "bf16" else d + 1
    if op == "weigh":
        old = sum(c for c, k in zip(ctx, t) if k > 0) if case["decay"] != 0.0 else 0
        return {"bytes": keys * hkv * (row + 4) + 4 * old * hkv + total * hq * (2 * d + 4), "flops": (2 * d + 3) * hq * pairs}
    kept = sum(min(k, case["keep"]) for k in t)
    looked = sum(k for k in t if k > case["keep"])
    return {"bytes": hkv * (4 * looked + kept * (2 * (2 * row + 4) + 4)), "flops": 0}


# ------------------------------------------------------------------------------------------------ 64 bits

def _power(e):
    """2^e in 64 bits, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _cached(s, name, places):
    """Rows of the pool at flat places (page, head, row) in 64 bits."""
    x = s[name]
    if s[name + "s"] is None:
        return x.view(-1, s["d"])[places].double()
    x = x.view(torch.uint8).view(-1, s["d"])[places].view(E4M3).double()
    return x * _power(s[name + "s"].view(-1)[places].to(torch.int64) - 127)[:, None]


def _flat(s, table, b, h, n):
    """Flat places of the positions 0 .. n - 1 of a head."""
    p = torch.arange(n)
    pg = table[b].cpu().long()[p // s["page"]]
    return ((pg * s["hkv"] + h) * s["page"] + p % s["page"]).cuda()


def _exact_rotate(s):
    out = []
    for x, w in ((s["Q"], s["qw"]), (s["K"], s["kw"])):
        y = x.double()
        if w is not None:
            norm = torch.sqrt((y * y).sum(-1, keepdim=True) / s["d"] + EPS)
            y = y / norm * w.double()
        if s["freq"] is not None and s["total"]:
            half = s["freq"].numel()
            pos = torch.cat([torch.arange(c, c + t) for c, t in zip(s["ctx_host"], s["t_host"])]).cuda().double()
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.outer(pos, s["freq"].double()))
            part = y[..., :2 * half].reshape(y.shape[0], y.shape[1], *((half, 2) if s["interleaved"] else (2, half)))
            part = part if s["interleaved"] else part.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn[:, None])
            z = z if s["interleaved"] else z.transpose(-1, -2)
            y = torch.cat((z.reshape(y.shape[0], y.shape[1], 2 * half), y[..., 2 * half:]), -1)
        out.append(y)
    return out


def _exact_prompt(s):
    G = s["hq"] // s["hkv"]
    O = torch.zeros((s["total"], s["hq"], s["d"]), dtype=torch.float64, device="cuda")
    LSE = torch.zeros((s["hq"], s["total"]), dtype=torch.float64, device="cuda")
    cu_q, cu_k = s["cu"].tolist(), s["cu_k"].tolist()
    for b in range(s["B"]):
        n = cu_k[b + 1] - cu_k[b]
        for h in range(s["hkv"]):
            K, V = (s[x][cu_k[b]:cu_k[b + 1], h].double() for x in ("K", "V"))
            for i0 in range(cu_q[b], cu_q[b + 1], 1024):  # 1024 queries at a time, with the keys the last of them sees
                i1 = min(i0 + 1024, cu_q[b + 1])
                last = torch.arange(i0, i1, device="cuda") + (n - cu_q[b + 1])
                m = i1 + n - cu_q[b + 1]
                z = torch.einsum("igd,jd->gij", s["Q"][i0:i1, h * G:(h + 1) * G].double(), K[:m]) / math.sqrt(s["d"])
                z = torch.where(torch.arange(m, device="cuda")[None, :] <= last[:, None], z, -math.inf)
                e = torch.logsumexp(z, -1)
                LSE[h * G:(h + 1) * G, i0:i1] = e
                O[i0:i1, h * G:(h + 1) * G] = torch.einsum("gij,jd->igd", torch.exp(z - e[..., None]), V[:m])
    return {"O": O, "LSE": LSE}


def _exact_weigh(s):
    G = s["hq"] // s["hkv"]
    out = s["out"].double().view(-1)
    cu = s["cu"].tolist()
    for b in range(s["B"]):
        n, c = s["ctx_host"][b] + cu[b + 1] - cu[b], s["ctx_host"][b]
        for h in range(s["hkv"] if cu[b + 1] > cu[b] else 0):
            at = _flat(s, s["table"], b, h, n)
            K = _cached(s, "k", at)
            got = torch.where(torch.arange(n, device="cuda") < c, s["w"].view(-1)[at].double() * s["decay"], 0.0)
            for i0 in range(cu[b], cu[b + 1], 512):
                i1 = min(i0 + 512, cu[b + 1])
                z = torch.einsum("igd,jd->igj", s["Q"][i0:i1, h * G:(h + 1) * G].double(), K) / math.sqrt(s["d"])
                p = torch.exp(z - s["LSE"][h * G:(h + 1) * G, i0:i1].t().double()[..., None])
                sees = torch.arange(n, device="cuda")[None, :] <= c + torch.arange(i0 - cu[b], i1 - cu[b], device="cuda")[:, None]
                got += torch.where(sees[:, None], p, 0.0).sum((0, 1))
            out[at] = got
    return out.view_as(s["out"])


def _exact_evict(s):
    kept = torch.full((s["B"], s["hkv"], s["keep"]), -1, dtype=torch.int32)
    new = {k: (s[k].view(torch.uint8) if s[k].dtype == E4M3 else s[k]).clone() for k in ("k", "v", "ks", "vs", "w") if s[k] is not None}
    for b in range(s["B"]):
        n = int(s["n"][b])
        m = min(n, s["keep"])
        for h in range(s["hkv"] if n else 0):
            at, to = _flat(s, s["table"], b, h, n), _flat(s, s["to"], b, h, m)
            w = s["w"].view(-1)[at].double()
            rank = w.clone()
            rank[:s["sink"]] = math.inf  # always kept, whatever their weight
            rank[n - s["recent"]:] = math.inf
            # the m-th largest, all above it, and of its equals the first
            limit = torch.topk(rank, m).values[-1]
            equal = rank == limit
            take = (rank > limit) | (equal & (torch.cumsum(equal, 0) <= m - (rank > limit).sum()))
            pos = torch.nonzero(take)[:, 0]
            kept[b, h, :m] = pos.cpu().to(torch.int32)
            for x, y in ((s[k], new[k]) for k in new):
                x = x.view(torch.uint8) if x.dtype == E4M3 else x
                wide = x.numel() // s["w"].numel()
                y.view(-1, wide)[to] = x.view(-1, wide)[at[pos]]
    return {"kept": kept, "lens": torch.clamp(s["n"], max=s["keep"])} | \
        {k: v.view(E4M3).double() if s[k].dtype == E4M3 else v.double() if s[k].is_floating_point() else v for k, v in new.items()}


def exact(case, seed):
    """From the definitions in 64 bits: head by head, with complex numbers for the rotation and ranks for the choice."""
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "prompt": _exact_prompt, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](s)
