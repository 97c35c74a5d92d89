"""The operators for prompts and bounded caches written down plainly in fp64, and the bounds the GPU's
results are held to.

Bounds (u = 2^-24, the half step of fp32; 2^-8 that of bf16):
* rotation: a cosine is off by 2^-22 (its angle by the rounding of a fraction of a turn to fp32, at most
  pi 2^-24, and the function's 2 units), and by position * frequency * 2^-51 for the product; the norm's
  sum of d squares, its root and three products are off by 32 u; the result rounds to bf16 once.
* attention: as in cache_ref.
* weights: score - LSE is an fp32 sum of d products and three terms of LSE / scale, in any order, so off by
  ds = (d + 16) u (B + |LSE|) with B = scale * sum |q_i k_i| (for an e4m3 cache also by what the query's two
  e4m3 terms may lose, as in cache_ref); LSE's split, its conversions and the scaling are off by 8 u (|s| + |LSE|),
  exp2 by 4 u; a sum of R rows is off by (R / 4 + 64) u at most.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from cache_ref import HALF_BF16, U, place, query_loss, rows_of


def bf16(r, shape, scale=1.0):
    return torch.from_numpy((r.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------------------------------------ rotation

def ref_rotate(x, w, freq, pos, eps, interleaved):
    """y and its bound for x [n, H, d] (fp64), positions [n]."""
    y = x.copy()
    if w is not None:
        y = y / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    out, size, far = y.copy(), np.abs(y), np.zeros_like(y)
    r = 0 if freq is None else len(freq)
    if r:
        t = pos[:, None].astype(np.float64) * freq[None].astype(np.float64)
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        ia, ib = (np.arange(0, 2 * r, 2), np.arange(1, 2 * r, 2)) if interleaved else (np.arange(r), np.arange(r, 2 * r))
        a, b = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
        far[..., ia] = far[..., ib] = np.abs(t)[:, None] * 2.0 ** -51
    tol = HALF_BF16 * np.abs(out) + size * (2.0 ** -22 + far + 32 * U) * (1 + HALF_BF16) + 2.0 ** -133
    return out, tol


# ------------------------------------------------------------------------------------------------ prompts

def ref_prompt(Q, K, V, cu_q, cu_k, scale, causal):
    """O, LSE and their bounds; rows outside every sequence are NaN in O (left as they were)."""
    total, Hq, d = Q.shape
    G = Hq // K.shape[1]
    O, tolO = np.full((total, Hq, d), np.nan), np.zeros((total, Hq, d))
    LSE, tolL = np.full((Hq, total), np.nan), np.zeros((Hq, total))
    for b in range(len(cu_q) - 1):
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(nq):
            seen = max(0, min(nk, i + nk - nq + 1)) if causal else nk
            for h in range(Hq):
                row = cu_q[b] + i
                if seen == 0:
                    O[row, h], LSE[h, row] = 0.0, -np.inf
                    continue
                q, Kh, Vh = Q[row, h], K[cu_k[b]:cu_k[b] + seen, h // G], V[cu_k[b]:cu_k[b] + seen, h // G]
                s = scale * (Kh @ q)
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                with np.errstate(invalid="ignore"):
                    O[row, h] = p @ Vh / l
                    A = p @ np.abs(Vh) / l
                LSE[h, row] = m + math.log(l)
                ds = d * U * scale * (np.abs(Kh) @ np.abs(q)).max() + 2 * U * np.abs(s).max()
                sums = (seen / 16 + 64) * U
                tolL[h, row] = ds + sums + 8 * U * (1 + abs(LSE[h, row]))
                tolO[row, h] = HALF_BF16 * np.abs(O[row, h]) + (HALF_BF16 + 4 * ds + 2 * sums + 8 * U) * A * (1 + HALF_BF16) + 1e-30
    return O, LSE, tolO, tolL


def hold_prompt(O, LSE, refs, finite=True):
    """Within the bounds where a row is in a sequence and finite there; the same infinities and NaN."""
    O_ref, LSE_ref, tolO, tolL = refs
    O, LSE = f64(O), f64(LSE)
    assert np.array_equal(np.isnan(O), np.isnan(O_ref))
    assert np.array_equal(np.where(np.isinf(O), O, 0), np.where(np.isinf(O_ref), O_ref, 0))
    assert np.array_equal(np.isneginf(LSE), np.isneginf(LSE_ref)) and np.array_equal(np.isnan(LSE), np.isnan(LSE_ref))
    ok = np.isfinite(O_ref)
    if finite:
        assert ok.any()
    past = np.max(np.abs(O[ok] - O_ref[ok]) - tolO[ok]) if ok.any() else 0.0
    assert past <= 0.0, f"O past its bound by {past:.3g}"
    assert np.all(O[np.isneginf(LSE_ref).T] == 0)
    ok = np.isfinite(LSE_ref)
    assert np.all(np.abs(LSE[ok] - LSE_ref[ok]) <= tolL[ok])


# ------------------------------------------------------------------------------------------------ weights

def ref_weigh(Q, LSE, k, ks, table, ctx, cu, page, scale, decay, w, out):
    """out (fp64, a copy of what the buffer held) and its bound: 0 where nothing is written."""
    out, tol = out.copy(), np.zeros(out.shape)
    d, hkv = Q.shape[2], k.shape[1]
    G = Q.shape[1] // hkv
    for b in range(len(cu) - 1):
        T = cu[b + 1] - cu[b]
        if T == 0:
            continue
        n = ctx[b] + T
        K = rows_of(k, ks, table, b, n, page)
        at = [place(table, b, p, page) for p in range(n)]
        pg, row = np.array([a[0] for a in at]), np.array([a[1] for a in at])
        see = np.arange(n)[None] <= ctx[b] + np.arange(T)[:, None]
        for h in range(hkv):
            old = np.where(np.arange(n) < ctx[b], decay * w[pg, h, row], 0.0) if decay != 0 else np.zeros(n)
            got, err = np.zeros(n), np.zeros(n)
            for g in range(G):
                q, L = Q[cu[b]:cu[b + 1], h * G + g], LSE[h * G + g, cu[b]:cu[b + 1]][:, None]
                s = scale * (q @ K[:, h].T)
                big = scale * (np.abs(q) @ np.abs(K[:, h]).T)
                lost = 0.0 if ks is None else scale * (np.stack([query_loss(x) for x in q]) @ np.abs(K[:, h]).T)
                with np.errstate(invalid="ignore", over="ignore"):
                    p = np.where(see & ~np.isneginf(L), np.exp(s - L), 0.0)
                    e = p * ((d + 16) * U * (big + np.abs(L)) + lost + 8 * U * (np.abs(s) + np.abs(L)) + 4 * U)
                got += p.sum(0)
                err += np.where(p > 0, e, 0.0).sum(0)
            out[pg, h, row] = old + got
            tol[pg, h, row] = 1.01 * err + (T * G / 4 + 64) * U * got + 4 * U * np.abs(old) + 1e-36
    return out, tol


# ------------------------------------------------------------------------------------------------ eviction

def ref_evict(pools, w, table, to, lens, keep, sink, recent, page):
    """kept, new lengths and the pools (k, v, ks, vs; None where there is none) and weights after packing."""
    B, hkv = len(lens), w.shape[1]
    new = [None if x is None else x.copy() for x in pools] + [w.copy()]
    kept = np.full((B, hkv, keep), -1, np.int64)
    for b in range(B):
        n = lens[b]
        src = [place(table, b, p, page) for p in range(n)]
        for h in range(hkv):
            pos = list(range(n))
            if n > keep:
                mid = pos[sink:n - recent]
                v = [-np.inf if np.isnan(w[src[p][0], h, src[p][1]]) else w[src[p][0], h, src[p][1]] for p in mid]
                best = sorted(range(len(mid)), key=lambda i: (-v[i], i))[:keep - sink - recent]
                pos = pos[:sink] + sorted(mid[i] for i in best) + pos[n - recent:]
            kept[b, h, :len(pos)] = pos
            for i, p in enumerate(pos):
                pg, row = place(to, b, i, page)
                for x, y in zip(list(pools) + [w], new):
                    if x is not None:
                        y[pg, h, row] = x[src[p][0], h, src[p][1]]
    return kept, np.minimum(lens, keep), new
