"""Plain 64-bit references of the paged cache's operators (CPU, numpy and
torch float64), and the tolerances they are compared with."""
from __future__ import annotations

import math

import numpy as np
import torch

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0


def ceil_div(a, b):
    return -(-a // b)


# ---- plan -------------------------------------------------------------------

def plan(cached, new, T, bs, table, free, count):
    """One request after the other.  Returns (table, free, seq, cu, slots,
    positions, count) with new tables."""
    table, free = np.array(table, dtype=np.int64), np.array(free, dtype=np.int64)
    mb, cap = table.shape[1], free.shape[0]
    cached = [min(max(int(c), 0), mb * bs) for c in cached]
    top = min(max(int(count), 0), cap)
    for b, n in enumerate(new):
        if n < 0:
            for j in range(ceil_div(cached[b], bs)):
                if top < cap:
                    free[top] = table[b, j]
                    top += 1
    have, wanted, used = top, 0, 0
    seq, cu = [], [0]
    slots, pos = np.full(T, -1, dtype=np.int64), np.full(T, -1, dtype=np.int64)
    for b, n in enumerate(new):
        m = max(int(n), 0)
        cu.append(cu[-1] + m)
        seq.append(0 if n < 0 else cached[b])
        if n < 0 or cached[b] + m > mb * bs or cu[-1] > T:
            continue
        old = ceil_div(cached[b], bs)
        more = ceil_div(cached[b] + m, bs) - old
        wanted += more
        if more and wanted > have:
            continue
        for j in range(more):
            table[b, old + j] = free[have - 1 - (wanted - more) - j]
        if more:
            used = wanted
        seq[b] = cached[b] + m
        for i in range(m):
            p = cached[b] + i
            slots[cu[b] + i] = table[b, p // bs] * bs + p % bs
            pos[cu[b] + i] = p
    return table, free, np.array(seq), np.array(cu), slots, pos, have - used


# ---- store --------------------------------------------------------------------

def stored(x, dtype, scale):
    """The element the pool holds for bf16 rows x [T, H, D] (a CPU tensor of
    the pool's dtype); scale [H] float32 or None."""
    if dtype != FP8:
        return x
    s = torch.ones(x.shape[1]) if scale is None else scale
    return (x.float() / s[:, None]).clamp(-FP8_MAX, FP8_MAX).to(FP8)


def store(x, pool, slots, scale):
    """pool (CPU, [nb, bs, H, D]) with the rows of x at their slots."""
    out = pool.clone()
    flat = out.view(torch.uint8 if pool.dtype == FP8 else pool.dtype).view(
        -1, pool.shape[2], pool.shape[3])
    src = stored(x, pool.dtype, scale)
    src = src.view(torch.uint8) if pool.dtype == FP8 else src
    for t, s in enumerate(slots):
        if 0 <= s < flat.shape[0]:
            flat[s] = src[t]
    return out


def bounds(pool, slots, before):
    """k_bounds after a store whose slots form the runs that a plan gives."""
    nb, bs = pool.shape[:2]
    out = before.clone()
    last = {}
    for s in slots:
        if 0 <= s < nb * bs:
            last[s // bs] = max(last.get(s // bs, -1), s % bs)
    for p, o in last.items():
        rows = pool[p, :o + 1].float()
        out[p, :, 0] = rows.amin(0).to(torch.bfloat16)
        out[p, :, 1] = rows.amax(0).to(torch.bfloat16)
    return out


# ---- selection ------------------------------------------------------------------

def select(q, k_bounds, bs, table, lens, keep, first, last):
    """int32 [B, H, keep] of CPU inputs."""
    B, Hq, D = q.shape
    nb, H = k_bounds.shape[:2]
    G = Hq // H
    sel = np.full((B, H, keep), -1, dtype=np.int64)
    kb = k_bounds.double().numpy()
    qd = q.double().numpy()
    for b in range(B):
        n = ceil_div(min(max(int(lens[b]), 0), table.shape[1] * bs), bs)
        for h in range(H):
            rank = []
            for j in range(n):
                page = int(table[b, j])
                if not 0 <= page < nb:
                    continue
                best = -math.inf
                for g in range(G):
                    qq = qd[b, h * G + g]
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = float((np.where(qq > 0, kb[page, h, 1], kb[page, h, 0]) * qq).sum())
                    if not math.isnan(s):
                        best = max(best, s)
                forced = j < first or j >= n - last
                rank.append((0 if forced else 1, 0.0 if forced else -best, j))
            got = sorted(j for _, _, j in sorted(rank)[:keep])
            sel[b, h, :len(got)] = got
    return sel


# ---- attention ------------------------------------------------------------------

def attention(q, k_cache, v_cache, table, lens, scale, k_scale=None, v_scale=None, window=0,
              sel=None):
    """(out, lse, tol_out, tol_lse) in float64, of CPU inputs.

    Tolerances, from the rounding steps the operator documents (u8 = 2^-8 is
    half a bf16 step, u24 half an fp32 one):
    * a logit is an fp32 sum of D exact products: off by at most
      d = (D + 4) u24 scale sum |q k|, and its softmax weight by 2 d
      relatively (numerator and sum), the exponential adding 2^-18;
    * each weight as two bf16 parts: u8^2 = 2^-16 relative, so with both the
      sum over V is off by (2^-16 + 2 d + 2^-18) sum p |v|, and its fp32
      accumulation by less than 2^-13 sum p |v| (n u24 for the n <= 2^11
      terms, two a key, of the tests' largest running chains);
    * the result rounded to bf16: u8 |out|, plus half the smallest subnormal.
    """
    B, Hq, D = q.shape
    nb, bs, H, _ = k_cache.shape
    G = Hq // H
    out = torch.zeros(B, Hq, D, dtype=torch.float64)
    tol = torch.zeros(B, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    tol_lse = torch.zeros(B, Hq, dtype=torch.float64)
    u8 = 2.0 ** -8
    ks = torch.ones(H) if k_scale is None else k_scale
    vs = torch.ones(H) if v_scale is None else v_scale
    kf = k_cache.float().double().reshape(nb * bs, H, D)
    vf = v_cache.float().double().reshape(nb * bs, H, D)
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * bs)
        lo = max(0, n - window) if window else 0
        for h in range(H):
            blocks = range(ceil_div(n, bs)) if sel is None else \
                [int(j) for j in sel[b, h] if 0 <= int(j) < ceil_div(n, bs)]
            rows = []
            for j in blocks:
                page = int(table[b, j])
                if 0 <= page < nb:
                    a, z = max(lo, j * bs), min(n, (j + 1) * bs)
                    rows += range(page * bs + a - j * bs, page * bs + z - j * bs) if z > a else []
            if not rows:
                continue
            k, v = kf[rows, h], vf[rows, h]
            qq = q[b, h * G:(h + 1) * G].double()
            f = scale * float(ks[h])
            z = qq @ k.T * f
            m = z.amax(1, keepdim=True)
            e = torch.exp(z - m)
            p = e / e.sum(1, keepdim=True)
            d = ((D + 4) * 2.0 ** -24 * abs(f) * (qq.abs() @ k.abs().T)).amax(1, keepdim=True)
            o = p @ v * float(vs[h])
            spread = p @ v.abs() * float(vs[h])
            out[b, h * G:(h + 1) * G] = o
            tol[b, h * G:(h + 1) * G] = (u8 * o.abs() + (2.0 ** -16 + 2 * d + 2.0 ** -18 + 2.0 ** -13)
                                         * spread + 2.0 ** -134)
            lse[b, h * G:(h + 1) * G] = (m + torch.log(e.sum(1, keepdim=True)))[:, 0]
            tol_lse[b, h * G:(h + 1) * G] = (2 * d + 2.0 ** -16 * (1 + m.abs()))[:, 0]
    return out, lse, tol, tol_lse
