"""Plain references of the paged cache's chunk attention and block upkeep
(CPU), and the chunk attention's tolerances."""
from __future__ import annotations

import math

import numpy as np
import torch

from pagedlib import ceil_div

FP8 = torch.float8_e4m3fn


# ---- chunk attention ----------------------------------------------------------

def chunk(q, k_cache, v_cache, table, cached, lens, cu, scale, k_scale=None, v_scale=None,
          window=0, before=None):
    """(out, lse, tol_out, tol_lse) in float64, of CPU inputs; rows of no
    request are as in ``before`` (NaN in lse).

    Tolerances, from the rounding steps that the operator documents (u8 = 2^-8
    is half a bf16 step relative to the value, u24 half an fp32 one, u11 half
    an fp16 one):
    * a logit is an fp32 sum of D exact products, scaled: off by at most
      d = (D + 4) u24 scale sum |q k|, and its softmax weight by 2 d
      relatively (numerator and sum), the exponential adding 2^-18;
    * each weight rounded once to bf16 (bf16 caches, u8) or fp16 (8-bit ones,
      u11, and at most 2^-39 of the largest where that is finer than fp16
      holds) for the product with V: the sum over V is off by u sum p |v|;
    * the fp32 sums over n keys by less than n u24 sum p |v|, for the weights'
      sum the same;
    * the result rounded to bf16: u8 |out|, plus half the smallest subnormal.
    """
    T, Hq, D = q.shape
    nb, bs, H, _ = k_cache.shape
    G = Hq // H
    u8, u24 = 2.0 ** -8, 2.0 ** -24
    fp8 = k_cache.dtype == FP8
    u = 2.0 ** -11 if fp8 else u8
    out = torch.zeros(T, Hq, D, dtype=torch.float64) if before is None else before.double()
    out = out.clone()
    tol = torch.zeros(T, Hq, D, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    tol_lse = torch.zeros(T, Hq, dtype=torch.float64)
    ks = torch.ones(H) if k_scale is None else k_scale
    vs = torch.ones(H) if v_scale is None else v_scale
    kf = k_cache.float().double().reshape(nb * bs, H, D)
    vf = v_cache.float().double().reshape(nb * bs, H, D)
    most = table.shape[1] * bs
    for b in range(table.shape[0]):
        r0 = min(max(int(cu[b]), 0), T)
        r1 = min(max(int(cu[b + 1]), r0), T)
        if r1 == r0:
            continue
        c = min(max(int(cached[b]), 0), most)
        n = min(max(int(lens[b]), 0), most)
        out[r0:r1] = 0
        lse[r0:r1] = -math.inf
        live = min(max(n - c, 0), r1 - r0)
        if not live:
            continue
        pos = np.arange(c + live)
        pages = np.asarray(table[b])[pos // bs]
        there = (pages >= 0) & (pages < nb)
        pos = pos[there]
        if not len(pos):
            continue
        rows = torch.as_tensor(pages[there] * bs + pos % bs)
        at = torch.arange(c, c + live)[:, None]
        p = torch.as_tensor(pos)[None, :]
        seen = p <= at
        if window:
            seen &= p > at - window
        count = seen.sum(1).double()[:, None]
        for h in range(H):
            # Keys that no row sees stay out of every product.
            k = kf[rows, h]
            v = vf[rows, h]
            for x in range(h * G, (h + 1) * G):
                qq = q[r0:r0 + live, x].double()
                f = scale * float(ks[h])
                z = (qq @ k.T * f).masked_fill(~seen, -math.inf)
                m = z.amax(1, keepdim=True)
                some = torch.isfinite(m)
                e = torch.where(some, torch.exp(z - torch.where(some, m, 0.0)), 0.0)
                s = e.sum(1, keepdim=True)
                w = torch.where(some, e / torch.where(s > 0, s, 1.0), 0.0)
                d = (D + 4) * u24 * abs(f) * (qq.abs() @ k.abs().T)
                d = torch.where(seen, d, 0.0).amax(1, keepdim=True)
                o = w @ v * float(vs[h])
                spread = w @ v.abs() * float(vs[h])
                out[r0:r0 + live, x] = o
                tol[r0:r0 + live, x] = (u8 * o.abs()
                                        + (u + 2 * d + 2.0 ** -18 + 2 * count * u24) * spread
                                        + 2.0 ** -134)
                if fp8:
                    tol[r0:r0 + live, x] += (2.0 ** -39 * torch.where(some, 1 / s, 0.0)
                                             * (seen.double() @ v.abs()) * float(vs[h]))
                lse[r0:r0 + live, x] = (m + torch.log(s))[:, 0]
                tol_lse[r0:r0 + live, x] = (2 * d + count * u24
                                            + 2.0 ** -16 * (1 + m.abs()))[:, 0]
    return out, lse, tol, tol_lse


# ---- upkeep ---------------------------------------------------------------------

def clamp(n, most):
    return min(max(int(n), 0), most)


def fork(parents, children, take, cached, bs, table, free, count, shares):
    """One pair after the other: (table, seq, src, dst, count, shares)."""
    table, shares = np.array(table, dtype=np.int64), np.array(shares, dtype=np.int64)
    B, mb = table.shape
    cached = [clamp(c, mb * bs) for c in cached]
    have = clamp(count, len(free))
    rows = [(int(p), int(c)) if 0 <= p < B and 0 <= c < B and p != c else None
            for p, c in zip(parents, children)]
    named = {r[0] for r in rows if r}
    seq, src, dst = list(cached), [-1] * len(rows), [-1] * len(rows)
    wanted, used, owned = 0, 0, set()
    old = table.copy()
    for i, r in enumerate(rows):
        if r is None:
            continue
        p, c = r
        first = c not in owned
        owned.add(c)
        if not first or c in named:
            continue
        n = cached[p] if take is None else clamp(take[i], cached[p])
        if n % bs:
            wanted += 1
            if wanted > have:
                continue
            used = wanted
            dst[i], src[i] = free[have - wanted], old[p, n // bs]
            table[c, n // bs] = dst[i]
        for j in range(n // bs):
            table[c, j] = old[p, j]
            if 0 <= old[p, j] < len(shares):
                shares[old[p, j]] += 1
        seq[c] = n
    return table, np.array(seq), np.array(src), np.array(dst), have - used, shares


def release(cached, keep, bs, table, free, count, shares):
    """(seq, count, free, shares)."""
    table, free = np.array(table), np.array(free, dtype=np.int64)
    held, shares = np.array(shares), np.array(shares, dtype=np.int64)
    most = table.shape[1] * bs
    top, freed, seq = clamp(count, len(free)), [], []
    for b in range(table.shape[0]):
        n = clamp(cached[b], most)
        m = clamp(keep[b], n)
        if m < n and m % bs:
            page = table[b, m // bs]
            if 0 <= page < len(held) and held[page] > 0:
                m = n
        seq.append(m)
        for j in range(ceil_div(m, bs), ceil_div(n, bs)):
            page = table[b, j]
            if 0 <= page < len(shares):
                if shares[page] <= 0:
                    freed.append(page)
                else:
                    shares[page] -= 1
    for page in sorted(set(freed), reverse=True):
        if top < len(free):
            free[top] = page
            top += 1
    return np.array(seq), top, free, shares


def compact(lens, bs, table, free, count, shares, limit):
    """(table, free, count, shares, remap, src, dst, moves)."""
    table, free = np.array(table, dtype=np.int64), np.array(free, dtype=np.int64)
    shares = np.array(shares, dtype=np.int64)
    nb, most = len(shares), table.shape[1] * bs
    gone = {int(x) for x in free[:clamp(count, len(free))] if 0 <= x < nb}
    remap = np.array([-1 if i in gone else i for i in range(nb)], dtype=np.int64)
    edge = min(max(limit, nb - len(gone)), nb)
    high = [i for i in range(edge, nb) if i not in gone]
    low = [i for i in range(edge) if i in gone]
    new = np.where(remap >= 0, shares, 0)
    for s, d in zip(high, low):
        remap[s] = d
        new[d], new[s] = shares[s], 0
    for b in range(table.shape[0]):
        for j in range(ceil_div(clamp(lens[b], most), bs)):
            if 0 <= table[b, j] < nb:
                table[b, j] = remap[table[b, j]]
    now = set(remap[remap >= 0].tolist())
    left = [i for i in range(nb - 1, -1, -1) if i not in now]
    free[:len(left)] = left
    pad = [-1] * (nb // 2 - len(high))
    return (table, free, len(left), new, remap, np.array(high + pad, dtype=np.int64),
            np.array(low[:len(high)] + pad, dtype=np.int64), len(high))
