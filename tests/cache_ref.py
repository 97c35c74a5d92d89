"""The paged cache and its attention written down plainly: fp64, one sequence, one head and one
token at a time, and the bounds the GPU's results are held to.

Bounds (u = 2^-24, the half step of fp32; 2^-8 that of bf16; L = the row's keys):
* a score's error is at most ds = d u B + 2 u |s|, B = scale * sum_i |q_i k_i| (fp32 sum of d
  exact products in any order, then the scaling); for an e4m3 cache also scale * sum_i e_i |k_i|
  with e_i what a query value's form may lose: with the row's largest in [1, 2) 2^E, either two
  e4m3 terms of q 2^(7 - E), off by half their least step 2^-9 where |q 2^(7 - E)| < 1/4 and
  exact above, or one f16 of q 2^-E, off by 2^-25 where |q 2^-E| < 2^-14;
* a probability is off by a factor exp(+-2 ds) (its score and the reference) and 4 u (exp2 and
  products), and rounds to bf16 once, 2^-8;
* l sums L terms in fp32 over 16 partial sums or more: (L / 16 + 64) u;
* O rounds to bf16 once, 2^-8 |O|; its sum over L keys adds (L / 16 + 64) u A with
  A = sum_j p_j |v_j| / l, and the probabilities' errors weigh in with A as well.
"""
from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8


def e4m3_round(y: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to even, by arithmetic; +-448 past the range, NaN stays."""
    y = np.asarray(y, np.float64)
    z = np.clip(y, -448.0, 448.0)
    _, e = np.frexp(z)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.clip(np.round(z / step) * step, -448.0, 448.0)


def quantise_row(x: np.ndarray):
    """(code values, scale code) of one row: e the least integer >= -126 with max |x| <= 448 * 2^e;
    every value a bf16."""
    x = np.asarray(x, np.float64)
    fine = np.abs(x[np.isfinite(x)])
    a = float(fine.max()) if fine.size else 0.0
    e = -126
    while a > 448.0 * 2.0 ** e:
        e += 1
    if e == 120:  # 2^128 is no bf16
        x = np.clip(x, -240 * 2.0 ** 120, 240 * 2.0 ** 120)
    with np.errstate(invalid="ignore"):
        return e4m3_round(x * 2.0 ** -e), e + 127


def place(table, b, pos, page):
    """(page, row) of a position."""
    return int(table[b][pos // page]), pos % page


def ref_write(K, V, k, v, ks, vs, table, cu, start, page):
    """In place on float64 arrays k, v (code values for an e4m3 cache) and integer ks, vs."""
    for b in range(len(cu) - 1):
        for i in range(cu[b + 1] - cu[b]):
            pg, row = place(table, b, start[b] + i, page)
            for h in range(k.shape[1]):
                for src, dst, sc in ((K, k, ks), (V, v, vs)):
                    x = src[cu[b] + i, h]
                    if sc is None:
                        dst[pg, h, row] = x
                    else:
                        dst[pg, h, row], sc[pg, h, row] = quantise_row(x)


def rows_of(c, sc, table, b, n, page):
    """fp64 [n, Hkv, d] rows of positions 0 .. n - 1."""
    out = []
    for p in range(n):
        pg, row = place(table, b, p, page)
        x = c[pg, :, row]
        out.append(x if sc is None else x * np.exp2(sc[pg, :, row].astype(np.float64) - 127.0)[:, None])
    return np.stack(out) if out else np.zeros((0,) + c.shape[1:2] + c.shape[3:])


def query_loss(q):
    """What a query row's values may lose in the form an e4m3 cache's kernels give them."""
    top = np.abs(q).max()
    if top == 0:
        return np.zeros_like(q)
    one = 2.0 ** math.floor(math.log2(top))
    rel = np.abs(q) / one
    return one * np.maximum(np.where(rel < 2.0 ** -9, 2.0 ** -17, 0.0), np.where(rel < 2.0 ** -14, 2.0 ** -25, 0.0))


def ref_tree(Q, k, v, ks, vs, table, ctx, cu, masks, page, scale):
    """O, LSE and their bounds (fp64): Q [total, Hq, d], caches as fp64."""
    total, Hq, d = Q.shape
    G = Hq // k.shape[1]
    O, A = np.zeros((total, Hq, d)), np.zeros((total, Hq, d))
    LSE, tolL = np.full((Hq, total), -np.inf), np.zeros((Hq, total))
    rel = np.zeros((total, Hq))
    for b in range(len(cu) - 1):
        T = cu[b + 1] - cu[b]
        if T == 0:
            continue
        n = ctx[b] + T
        K, V = rows_of(k, ks, table, b, n, page), rows_of(v, vs, table, b, n, page)
        for i in range(T):
            word = (1 << (i + 1)) - 1 if masks is None else int(masks[cu[b] + i])
            see = [j for j in range(n) if j < ctx[b] or (word >> (j - ctx[b])) & 1]
            if not see:
                continue
            for h in range(Hq):
                q, Kh, Vh = Q[cu[b] + i, h], K[see, h // G], V[see, h // G]
                s = scale * (Kh @ q)
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                with np.errstate(invalid="ignore"):
                    O[cu[b] + i, h] = p @ Vh / l
                    A[cu[b] + i, h] = p @ np.abs(Vh) / l
                LSE[h, cu[b] + i] = m + math.log(l)
                big = scale * (np.abs(Kh) @ np.abs(q)).max()
                ds = d * U * big + 2 * U * np.abs(s).max()
                if ks is not None:
                    ds += scale * (np.abs(Kh) @ query_loss(q)).max()
                sums = (len(see) / 16 + 64) * U
                tolL[h, cu[b] + i] = ds + sums + 8 * U * (1 + abs(LSE[h, cu[b] + i]))
                rel[cu[b] + i, h] = HALF_BF16 + 2 * (2 * ds) + 2 * sums + 8 * U
    return O, LSE, HALF_BF16 * np.abs(O) + rel[..., None] * A * (1 + HALF_BF16) + 1e-30, tolL


def hold(O, LSE, refs):
    """O, LSE (tensors) within the bounds of ref_tree's result."""
    O_ref, LSE_ref, tolO, tolL = refs
    O, LSE = O.double().cpu().numpy(), LSE.double().cpu().numpy()
    dead = np.isneginf(LSE_ref)
    assert np.array_equal(np.isneginf(LSE), dead)
    assert not np.isnan(LSE).any() and not np.isnan(O).any()
    assert np.all(O[dead.T] == 0)
    worst = np.max(np.abs(O - O_ref) / tolO) if O.size else 0.0
    assert worst <= 1.0, f"O off by {worst:.3g} of its bound"
    with np.errstate(invalid="ignore"):
        e = np.where(dead, 0.0, np.abs(LSE - LSE_ref) - tolL)
    assert np.all(e <= 0.0), f"LSE past its bound by {e.max():.3g}"


class Batch:
    """A cache with random pages, its tokens and the tensors a call takes.  Everything the
    sequences do not own (other pages, rows past their ends) holds NaN."""

    def __init__(self, seed, hkv, G, d, page, f8, ctx, T, *, masks="tree", extra=2, pad_q=0, scale=None, gap=0):
        r = np.random.default_rng(seed)
        self.hkv, self.G, self.d, self.page, self.f8 = hkv, G, d, page, f8
        self.ctx, self.T = list(ctx), list(T)
        B = len(self.ctx)
        self.scale = 1.0 / math.sqrt(d) if scale is None else scale
        need = [-(-(c + t) // page) for c, t in zip(ctx, T)]
        P = sum(need) + extra
        self.max_pages = max(need + [1])
        order = r.permutation(P)
        self.table = np.full((B, self.max_pages), 2 ** 31 - 1, np.int64)  # entries nobody needs: far outside
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cu = [gap]
        for t in self.T:
            self.cu.append(self.cu[-1] + t)
        self.total = self.cu[-1] + pad_q
        bf = lambda a: torch.from_numpy(a).to(torch.bfloat16)  # noqa: E731
        k, v = (bf(r.standard_normal((P, hkv, page, d)).astype(np.float32)) for _ in range(2))
        own = np.zeros((P, page), bool)
        for b in range(B):
            for p in range(self.ctx[b] + self.T[b]):
                pg, row = place(self.table, b, p, page)
                own[pg, row] = True
        stale = torch.from_numpy(~own)[:, None, :].expand(P, hkv, page)
        if f8:
            self.k, self.v, self.ks, self.vs = [], [], None, None
            for x, name in ((k, "k"), (v, "v")):
                rows = x.double().numpy().reshape(-1, d)
                codes, sc = zip(*[quantise_row(row) for row in rows]) if len(rows) else ((), ())
                c = torch.from_numpy(np.array(codes, np.float32).reshape(P, hkv, page, d)).to(torch.float8_e4m3fn)
                u = c.view(torch.uint8)
                u[stale] = 0x7F
                s = torch.from_numpy(np.array(sc, np.uint8).reshape(P, hkv, page))
                s[stale] = 255
                setattr(self, name, c)
                setattr(self, name + "s", s)
        else:
            k[stale] = float("nan")
            v[stale] = float("nan")
            self.k, self.v, self.ks, self.vs = k, v, None, None
        self.Q = bf(r.standard_normal((self.total, hkv * G, d)).astype(np.float32))
        if masks == "chain":
            self.masks = None
        else:
            words = np.zeros(self.total, np.uint64)
            for b, t in enumerate(self.T):
                for i in range(t):
                    if masks == "none":
                        w = 0
                    elif masks == "random":  # any bits, also those past the sequence's tokens
                        w = int(r.integers(0, 2 ** 63)) * 2 + int(r.integers(0, 2))
                    else:
                        up = int(r.integers(-1, i)) if i else -1
                        w = (1 << i) | (int(words[self.cu[b] + up]) if up >= 0 else 0)
                    words[self.cu[b] + i] = w
            self.masks = words

    def dev(self, device="cuda"):
        """The call's tensors: positional arguments after Q and keyword arguments."""
        t = lambda a: torch.as_tensor(np.asarray(a, np.int32), device=device)  # noqa: E731
        kw = dict(scale=self.scale)
        if self.masks is not None:
            kw["tree_mask"] = torch.from_numpy(self.masks.view(np.int64)).to(device)
        if self.f8:
            kw.update(k_scale=self.ks.to(device), v_scale=self.vs.to(device))
        return [self.Q.to(device), self.k.to(device), self.v.to(device), t(self.table).reshape(len(self.ctx), -1),
                t(self.ctx), t(self.cu), max(self.T + [1])], kw

    def reference(self):
        f = lambda x: x.double().numpy()  # noqa: E731
        ks, vs = (None, None) if not self.f8 else (self.ks.numpy(), self.vs.numpy())
        return ref_tree(f(self.Q), f(self.k), f(self.v), ks, vs, self.table, self.ctx, self.cu, self.masks, self.page,
                        self.scale)
