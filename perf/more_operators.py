"""Cases of the paged key-value cache's operators for many new tokens per
request and for the upkeep of its blocks, for measurement.

``attention_chunk_paged`` lets several new tokens of each request attend over
the cache that already holds them (prompts, chunks of prompts, drafts to be
verified).  ``paged_fork`` gives a request's blocks to further rows of the
block table, ``paged_free`` takes rows or the ends of rows back, and
``paged_compact`` moves what is in use to the low end of the pool;
``paged_copy`` moves the contents that a fork or a compaction names, once a
layer.

``own`` false: the operators in elementary torch operations.  ``own`` true:
the library's kernels through ``mixture_value_projection_amd.binding``.
"""
import math

import torch

own = False

DEV = "cuda"
FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # One user's short question after a short prompt: all latency.
        dict(name="chunk_short", op="attend", dtype="bf16", batch=1, heads=32, kv_heads=8,
             head_dim=128, block=16, fewest=19, most=19, shortest=130, longest=130, window=0,
             refused=False, padding=0),
        # Four drafted tokens verified in each request of the serving batch.
        dict(name="chunk_drafts", op="attend", dtype="bf16", batch=64, heads=32, kv_heads=8,
             head_dim=128, block=16, fewest=4, most=4, shortest=500, longest=8000, window=0,
             refused=False, padding=0),
        # A whole prompt at once, nothing cached before.
        dict(name="chunk_prompt", op="attend", dtype="bf16", batch=1, heads=32, kv_heads=8,
             head_dim=128, block=16, fewest=8192, most=8192, shortest=0, longest=0, window=0,
             refused=False, padding=0),
        # The last chunk of a long document.
        dict(name="chunk_long", op="attend", dtype="bf16", batch=1, heads=32, kv_heads=8,
             head_dim=128, block=64, fewest=2048, most=2048, shortest=129024, longest=129024,
             window=0, refused=False, padding=0),
        # Running requests and chunks of prompts in one batch, 8-bit cache, one
        # request refused by the plan, rows behind the last token.
        dict(name="chunk_mixed_fp8", op="attend", dtype="fp8", batch=24, heads=32, kv_heads=8,
             head_dim=128, block=32, fewest=1, most=1500, shortest=0, longest=16000, window=0,
             refused=True, padding=61),
        # Another layer shape: narrow heads, a group of 5, a block size that is
        # no power of two, a sliding window.
        dict(name="chunk_odd", op="attend", dtype="bf16", batch=37, heads=15, kv_heads=3,
             head_dim=64, block=24, fewest=1, most=601, shortest=0, longest=6001, window=2500,
             refused=True, padding=7),
        # Eight answers to each of eight prompts begin: rows and, for one layer,
        # the last blocks' contents.
        dict(name="fork_answers", op="fork", dtype="bf16", parents=8, children=56, kv_heads=8,
             head_dim=128, block=16, shortest=500, longest=8000, short_of=0, spare=300),
        # Rows of very long documents forked, the pool nearly used up.
        dict(name="fork_long_fp8", op="fork", dtype="fp8", parents=3, children=12, kv_heads=8,
             head_dim=128, block=32, shortest=20000, longest=200000, short_of=3, spare=7),
        # After a step with drafts: some requests end, the others drop what was
        # not accepted.
        dict(name="free_step", op="free", requests=64, ending=5, shared=0, block=16,
             shortest=20, longest=8000, cut=6, spare=40),
        # Many answers that share their prompts' blocks end at once.
        dict(name="free_shared", op="free", requests=203, ending=150, shared=120, block=16,
             shortest=200, longest=12000, cut=40, spare=400),
        # A small pool's blocks moved together.
        dict(name="compact_small", op="compact", dtype="bf16", requests=21, kv_heads=8,
             head_dim=128, block=16, shortest=40, longest=3000, holes=700, shared=3, limit=0),
        # A large pool to be cut to a given size.
        dict(name="compact_large_fp8", op="compact", dtype="fp8", requests=150, kv_heads=8,
             head_dim=128, block=32, shortest=300, longest=12000, holes=9000, shared=20,
             limit=14500),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "fork", "free", "compact"])
    dtype = rng.choice(["bf16", "bf16", "fp8"])
    kv_heads = rng.choice([1, 2, 3, 4, 6, 8, 8])
    group = rng.choice([1, 2, 3, 4, 4, 5, 8, 16])
    head_dim = rng.choice([64, 128, 128, 128, 256])
    block = rng.choice([8, 16, 16, 24, 32, 48, 64, 128])
    if op == "attend":
        batch = _log(rng, 1, 100)
        # Products stay below the longest listed case's, and so do keys read.
        width = batch * kv_heads * head_dim
        most = _log(rng, 1, max(1, min(8192, 2 ** 29 // (width * group),
                                       int((2 ** 39 / (width * group)) ** 0.5))))
        longest = _log(rng, 1, max(1, min(131072, 400000 * 1024 // width,
                                          2 ** 39 // (width * group * most))))
        return dict(op=op, dtype=dtype, batch=batch, heads=kv_heads * group, kv_heads=kv_heads,
                    head_dim=head_dim, block=block, fewest=_log(rng, 1, most), most=most,
                    shortest=rng.choice([0, _log(rng, 1, longest)]), longest=longest,
                    window=rng.choice([0, 0, 0, _log(rng, 1, longest + most)]),
                    refused=rng.random() < 0.3, padding=rng.choice([0, rng.randint(1, 63)]))
    requests = _log(rng, 1, 300)
    if op == "fork":
        parents = _log(rng, 1, 100)
        longest = _log(rng, 1, max(1, min(200000, 300000 * 1024 // (parents * kv_heads * head_dim))))
        return dict(op=op, dtype=dtype, parents=parents, children=_log(rng, 1, 200),
                    kv_heads=kv_heads, head_dim=head_dim, block=block,
                    shortest=_log(rng, 1, longest), longest=longest,
                    short_of=rng.choice([0, 0, rng.randint(1, 4)]), spare=_log(rng, 1, 500))
    if op == "free":
        longest = _log(rng, 1, 12000)
        ending = rng.randint(0, requests)
        return dict(op=op, requests=requests, ending=ending, shared=rng.randint(0, requests - 1),
                    block=block, shortest=_log(rng, 1, longest), longest=longest,
                    cut=_log(rng, 1, 50), spare=_log(rng, 1, 500))
    longest = _log(rng, 1, max(1, min(12000, 400000 * 1024 // (requests * kv_heads * head_dim))))
    blocks = requests * -(-longest // block)
    return dict(op=op, dtype=dtype, requests=requests, kv_heads=kv_heads, head_dim=head_dim,
                block=block, shortest=_log(rng, 1, longest), longest=longest,
                holes=_log(rng, 1, max(1, min(9000, blocks))), shared=rng.randint(0, requests - 1),
                limit=rng.choice([0, 0, blocks // 2]))


# ---- lengths, the same for every seed -----------------------------------------

def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], even in their logarithm, in mixed order."""
    out = []
    for i in range(n):
        u = (0.31 + i * 0.6180339887498949) % 1.0
        out.append(min(hi, max(lo, int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** u)) - 1)))
    return out


def _blocks(n, block):
    return (n + block - 1) // block


def _chunks(case):
    """Per request: cached tokens, new tokens, tokens after the plan."""
    n = case["batch"]
    cached = _spread(n, case["shortest"], case["longest"])
    cached[0] = case["longest"]
    # From the other end, so that long chunks meet short caches too.
    new = _spread(n, case["fewest"], case["most"])[::-1]
    new[-1] = case["most"]
    total = [c + m for c, m in zip(cached, new)]
    if case["refused"] and n > 1:
        total[n // 2] = cached[n // 2]  # its tokens got no slots
    return cached, new, total


def _fork_plan(case):
    """Parents' lengths, and per pair its parent and the tokens it takes over."""
    lens = _spread(case["parents"], case["shortest"], case["longest"])
    lens[0] = case["longest"]
    parent = [i % case["parents"] for i in range(case["children"])]
    # Every third pair takes a prefix only.
    take = [lens[p] if i % 3 else max(1, lens[p] * 5 // 8) for i, p in enumerate(parent)]
    return lens, parent, take


def _free_plan(case):
    """Per row: tokens, tokens kept, and the row whose prompt it shares (-1)."""
    n, bs = case["requests"], case["block"]
    lens = _spread(n, case["shortest"], case["longest"])
    lens[0] = case["longest"]
    step = n / max(case["ending"], 1)
    ends = {int(i * step) for i in range(case["ending"])}
    of = [-1] * n
    for i in range(case["shared"]):
        b = 1 + i % max(n - 1, 1)
        if n > 1 and of[b] < 0:
            of[b] = 0 if b < 8 else (b % 7)
    of[:7] = [-1] * min(7, n)
    keep = []
    for b in range(n):
        if b in ends:
            keep.append(0)
        else:
            # Back by some tokens, never into the shared part.
            held = _common(lens, of, b, bs) * bs if of[b] >= 0 else 0
            others = [_common(lens, of, x, bs) * bs for x in range(n) if of[x] == b]
            keep.append(max([0, held, lens[b] - (b * 7) % (case["cut"] + 1)] + others))
    return lens, keep, of


def _common(lens, of, b, bs):
    """Full blocks that row b shares with the row it was forked from."""
    return min(lens[b], lens[of[b]]) * 3 // 4 // bs


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def _pool(g, num_blocks, block, heads, dim, dtype, scale, lean):
    """Cache rows: normal, and for keys (lean > 0) with a part that the
    tokens of a block share, as neighbouring tokens do."""
    x = torch.empty(num_blocks, block, heads, dim, dtype=FP8 if dtype == "fp8" else torch.bfloat16,
                    device=DEV)
    step = max(1, (1 << 27) // (block * heads * dim))
    for i in range(0, num_blocks, step):
        n = min(step, num_blocks - i)
        r = _rows(g, n, block, heads, dim)
        if lean:
            r = r + lean * _rows(g, n, 1, heads, dim)
        if dtype == "fp8":
            x[i:i + n] = (r / scale[None, None, :, None]).clamp(-FP8_MAX, FP8_MAX).to(FP8)
        else:
            x[i:i + n] = r.to(torch.bfloat16)
    return x


def _pools(st, g, case, num_blocks):
    H, D, bs = case["kv_heads"], case["head_dim"], case["block"]
    st["k_scale"] = st["v_scale"] = None
    if case["dtype"] == "fp8":
        st["k_scale"] = (1.0 + torch.rand(H, generator=g, device=DEV)) / 64.0
        st["v_scale"] = (1.0 + torch.rand(H, generator=g, device=DEV)) / 64.0
    st["k"] = _pool(g, num_blocks, bs, H, D, case["dtype"], st["k_scale"], 1.0)
    st["v"] = _pool(g, num_blocks, bs, H, D, case["dtype"], st["v_scale"], 0.0)


def _rows_of_table(need, perm, width):
    """A block table whose rows take their blocks from perm in turn."""
    table = torch.full((len(need), width), -1, dtype=torch.int32, device=DEV)
    col = torch.arange(width, device=DEV)
    held = col < _ints(need, torch.int64)[:, None]
    table[held] = perm[:int(sum(need))]
    return table


def _stack(left, capacity):
    free = torch.full((capacity,), -1, dtype=torch.int32, device=DEV)
    free[:left.numel()] = left
    return free, _ints([left.numel()])


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    bs = case["block"]

    def shuffled(n):
        return torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    if case["op"] == "attend":
        cached, new, total = _chunks(case)
        st["cached"], st["seq"] = _ints(cached), _ints(total)
        cu = [0]
        for m in new:
            cu.append(cu[-1] + m)
        st["cu"], st["rows"] = _ints(cu), cu
        need = [_blocks(n, bs) for n in total]
        pool = sum(need) + 3
        st["table"] = _rows_of_table(need, shuffled(pool), max(1, max(need)))
        _pools(st, g, case, pool)
        st["q"] = _rows(g, cu[-1] + case["padding"], case["heads"],
                        case["head_dim"]).to(torch.bfloat16)
        # Rows behind the last token keep what the output held before.
        st["out"] = torch.zeros_like(st["q"])
    elif case["op"] == "fork":
        lens, parent, take = _fork_plan(case)
        P, n = case["parents"], case["children"]
        need = [_blocks(x, bs) for x in lens] + [0] * n
        parts = sum(1 for t in take if t % bs)
        held = sum(need)
        pool = held + case["spare"] + max(0, parts - case["short_of"])
        perm = shuffled(pool)
        st["table"] = _rows_of_table(need, perm, max(need) + 8)
        # With short_of the stack holds too few for the last pairs; the others
        # of the pool are somebody else's.
        st["free"], st["count"] = _stack(
            perm[held:held + max(0, parts - case["short_of"])] if case["short_of"] else perm[held:],
            pool)
        st["cached"] = _ints(lens + [0] * n)
        st["parents"], st["children"] = _ints(parent), _ints([P + i for i in range(n)])
        st["take"] = _ints(take)
        st["shares"] = torch.zeros(pool, dtype=torch.int32, device=DEV)
        _pools(st, g, case, pool)
        st["bounds"] = _rows(g, pool, case["kv_heads"], 2, case["head_dim"]).to(torch.bfloat16)
    elif case["op"] == "free":
        lens, keep, of = _free_plan(case)
        common = [_common(lens, of, b, bs) if of[b] >= 0 else 0 for b in range(len(lens))]
        need = [_blocks(x, bs) for x in lens]
        pool = sum(need) + case["spare"]
        perm = shuffled(pool)
        width = max(need) + 8
        st["table"] = _rows_of_table(need, perm, width)
        st["shares"] = torch.zeros(pool, dtype=torch.int32, device=DEV)
        unused = [perm[sum(need):]]
        for b, c in enumerate(common):
            if c:
                unused.append(st["table"][b, :c].clone())
                st["table"][b, :c] = st["table"][of[b], :c]
                st["shares"][st["table"][b, :c].long()] += 1
        st["free"], st["count"] = _stack(torch.cat(unused), pool)
        st["cached"], st["keep"] = _ints(lens), _ints(keep)
    else:
        n = case["requests"]
        lens = _spread(n, case["shortest"], case["longest"])
        lens[0] = case["longest"]
        need = [_blocks(x, bs) for x in lens]
        pool = sum(need) + case["holes"]
        perm = shuffled(pool)
        st["table"] = _rows_of_table(need, perm, max(need) + 8)
        st["shares"] = torch.zeros(pool, dtype=torch.int32, device=DEV)
        unused = [perm[sum(need):]]
        for b in range(n - case["shared"], n):
            c = min(lens[0], lens[b]) * 3 // 4 // bs
            if b and c:
                unused.append(st["table"][b, :c].clone())
                st["table"][b, :c] = st["table"][0, :c]
                st["shares"][st["table"][0, :c].long()] += 1
        st["free"], st["count"] = _stack(torch.cat(unused), pool)
        st["cached"] = _ints(lens)
        _pools(st, g, case, pool)
        st["bounds"] = _rows(g, pool, case["kv_heads"], 2, case["head_dim"]).to(torch.bfloat16)
    return st


# ---- one pass -----------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return {"attend": _own_attend, "fork": _own_fork, "free": _own_free,
                "compact": _own_compact}[op](st)
    return {"attend": _attend, "fork": _fork, "free": _free, "compact": _compact}[op](st)


def _own_attend(st):
    from mixture_value_projection_amd import binding
    case = st["case"]
    return binding.attention_chunk_paged(st["q"], st["k"], st["v"], st["table"], st["cached"],
                                         st["seq"], st["cu"], case["head_dim"] ** -0.5,
                                         k_scale=st["k_scale"], v_scale=st["v_scale"],
                                         window=case["window"], out=st["out"])


def _own_fork(st):
    from mixture_value_projection_amd import binding
    # The share counts are updated in place: a pass works on its own.
    shares = st["shares"].clone()
    f = binding.paged_fork(st["parents"], st["children"], st["case"]["block"], st["table"],
                           st["cached"], st["free"], st["count"], shares, fork_lens=st["take"])
    binding.paged_copy(f.copy_src, f.copy_dst, st["k"], st["v"], k_bounds=st["bounds"])
    return [st["table"], f.seq_lens, f.copy_src, f.copy_dst, f.free_count, shares, st["k"],
            st["v"], st["bounds"]]


def _own_free(st):
    from mixture_value_projection_amd import binding
    shares = st["shares"].clone()
    f = binding.paged_free(st["cached"], st["keep"], st["case"]["block"], st["table"], st["free"],
                           st["count"], shares)
    return [f.seq_lens, f.free_count, st["free"], shares]


def _own_compact(st):
    from mixture_value_projection_amd import binding
    c = binding.paged_compact(st["cached"], st["case"]["block"], st["table"], st["free"],
                              st["count"], st["shares"], limit=st["case"]["limit"],
                              block_table_out=torch.empty_like(st["table"]),
                              free_blocks_out=torch.empty_like(st["free"]),
                              shares_out=torch.empty_like(st["shares"]))
    binding.paged_copy(c.move_src, c.move_dst, st["k"], st["v"], k_bounds=st["bounds"],
                       count=c.move_count)
    return [c.block_table, c.free_blocks, c.free_count, c.shares, c.remap, c.move_src, c.move_dst,
            c.move_count, st["k"], st["v"], st["bounds"]]


# ---- the plain forms ------------------------------------------------------------

def _attend(st):
    case = st["case"]
    H, D, bs, w = case["kv_heads"], case["head_dim"], case["block"], case["window"]
    G = case["heads"] // H
    cached, new, total = _chunks(case)
    out = st["out"]
    scale = D ** -0.5
    if st["k_scale"] is not None:
        scale = (st["k_scale"] * scale)[:, None, None]
    for b, n in enumerate(total):
        c, rows = cached[b], n - cached[b]
        if rows < new[b]:
            out[st["rows"][b]:st["rows"][b + 1]] = 0
            continue
        lo = max(0, c + 1 - w) if w else 0
        ids = st["table"][b, lo // bs:_blocks(n, bs)].long()
        first = lo // bs * bs
        k = st["k"][ids].reshape(-1, H, D)[lo - first:n - first].float().transpose(0, 1)
        v = st["v"][ids].reshape(-1, H, D)[lo - first:n - first].float().transpose(0, 1)
        k, v = k.contiguous(), v.contiguous()
        p = torch.arange(lo, n, device=DEV)
        step = max(1, (1 << 30) // (case["heads"] * (n - lo)))
        for i in range(0, rows, step):
            m = min(step, rows - i)
            t = st["rows"][b] + i
            q = st["q"][t:t + m].float().reshape(m, H, G, D).permute(1, 2, 0, 3)
            s = torch.matmul(q.reshape(H, G * m, D), k.transpose(1, 2)) * scale
            at = torch.arange(c + i, c + i + m, device=DEV)[:, None]
            seen = p <= at
            if w:
                seen = seen & (p > at - w)
            s = s.reshape(H, G, m, -1).masked_fill_(~seen, -math.inf)
            s = torch.exp(s - s.amax(-1, keepdim=True))
            s = s / s.sum(-1, keepdim=True)
            o = torch.matmul(s.reshape(H, G * m, -1), v)
            if st["v_scale"] is not None:
                o = o * st["v_scale"][:, None, None]
            out[t:t + m] = o.reshape(H, G, m, D).permute(2, 0, 1, 3).reshape(
                m, case["heads"], D).to(torch.bfloat16)
    return out


def _raw(pool):
    return pool.view(torch.uint8) if pool.dtype == FP8 else pool


def _copied(st, src, dst):
    for pool in (st["k"], st["v"], st["bounds"]):
        _raw(pool)[dst] = _raw(pool)[src]


def _fork(st):
    bs, table = st["case"]["block"], st["table"]
    parents, children = st["parents"].long(), st["children"].long()
    size = torch.minimum(st["take"].long().clamp(min=0), st["cached"].long()[parents])
    full, part = size // bs, size % bs > 0
    upto = part.long().cumsum(0)
    have = st["count"].long()
    ok = ~part | (upto <= have)
    new = torch.where(ok & part, st["free"].long()[(have - upto).clamp(min=0)], -1)
    col = torch.arange(table.shape[1], device=DEV)
    shared = (col < full[:, None]) & ok[:, None]
    ids = table[parents]
    last = ids.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    table[children] = torch.where(shared, ids, table[children])
    took = torch.nonzero(new >= 0)[:, 0]
    table[children[took], full[took]] = new[took].to(torch.int32)
    used = ids[shared].long()
    shares = st["shares"] + torch.bincount(used, minlength=st["shares"].numel()).to(torch.int32)
    src = torch.where(new >= 0, last, -1)
    seq = st["cached"].clone()
    seq[children] = torch.where(ok, size.to(torch.int32), seq[children])
    _copied(st, src[took].long(), new[took])
    return [table, seq, src, new.to(torch.int32), (have - torch.minimum(upto[-1:], have)).to(torch.int32),
            shares, st["k"], st["v"], st["bounds"]]


def _free(st):
    bs, table = st["case"]["block"], st["table"]
    cached = st["cached"].long()
    keep = torch.minimum(st["keep"].long().clamp(min=0), cached)
    # A row is not cut inside a block that others hold too.
    last = table.gather(1, (keep // bs).clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    stays = (keep % bs > 0) & (keep < cached) & (st["shares"][last.clamp(min=0)] > 0) & (last >= 0)
    keep = torch.where(stays, cached, keep)
    col = torch.arange(table.shape[1], device=DEV)
    goes = (col >= _blocks(keep, bs)[:, None]) & (col < _blocks(cached, bs)[:, None])
    n = torch.bincount(table[goes].long(), minlength=st["shares"].numel())
    freed = n > st["shares"]
    shares = (st["shares"] - n.to(torch.int32)).clamp(min=0)
    ids = torch.nonzero(freed)[:, 0].flip(0).to(torch.int32)
    count = st["count"].long()
    st["free"][count + torch.arange(ids.numel(), device=DEV)] = ids
    return [keep.to(torch.int32), (count + ids.numel()).to(torch.int32), st["free"], shares]


def _compact(st):
    case = st["case"]
    nb, bs, table = st["shares"].numel(), case["block"], st["table"]
    ids = torch.arange(nb, device=DEV)
    live = torch.ones(nb, dtype=torch.bool, device=DEV)
    live[st["free"].long()[:int(st["count"])]] = False
    edge = torch.clamp(live.sum(), min=case["limit"])
    src = torch.nonzero(live & (ids >= edge))[:, 0]
    dst = torch.nonzero(~live & (ids < edge))[:, 0][:src.numel()]
    src = src[:dst.numel()]
    remap = torch.where(live, ids, -1)
    remap[src] = dst
    used = torch.arange(table.shape[1], device=DEV) < _blocks(st["cached"].long(), bs)[:, None]
    used = used & (table >= 0)
    new_table = torch.where(used, remap[table.long().clamp(min=0)], table).to(torch.int32)
    now = live.clone()
    now[src], now[dst] = False, True
    shares = torch.where(now, st["shares"], 0)
    shares[dst] = st["shares"][src]
    left = torch.nonzero(~now)[:, 0].flip(0)
    free = st["free"].clone()
    free[:left.numel()] = left.to(torch.int32)
    moves = [torch.full((nb // 2,), -1, dtype=torch.int32, device=DEV) for _ in range(2)]
    moves[0][:src.numel()], moves[1][:src.numel()] = src.to(torch.int32), dst.to(torch.int32)
    _copied(st, src, dst)
    return [new_table, free, _ints([left.numel()]), shares, remap.to(torch.int32), moves[0],
            moves[1], _ints([src.numel()]), st["k"], st["v"], st["bounds"]]


# ---- the definitions in 64 bits ---------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"attend": _exact_attend, "fork": _exact_fork, "free": _exact_free,
            "compact": _exact_compact}[case["op"]](case, st)


def _wide(t):
    return t.float().double()


def _exact_attend(case, st):
    H, D, bs, w = case["kv_heads"], case["head_dim"], case["block"], case["window"]
    G = case["heads"] // H
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    cached, new, total = _chunks(case)
    for b, n in enumerate(total):
        if n < cached[b] + new[b]:
            continue
        p = torch.arange(n, device=DEV)
        page = st["table"][b].long()[p // bs]
        for h in range(H):
            k, v = _wide(st["k"][page, p % bs, h]), _wide(st["v"][page, p % bs, h])
            if case["dtype"] == "fp8":
                k, v = k * _wide(st["k_scale"])[h], v * _wide(st["v_scale"])[h]
            for i in range(0, new[b], 1024):
                m = min(1024, new[b] - i)
                at = torch.arange(cached[b] + i, cached[b] + i + m, device=DEV)
                hidden = p[None, :] > at[:, None]
                if w:
                    hidden |= p[None, :] + w <= at[:, None]
                t = st["rows"][b] + i
                for x in range(h * G, (h + 1) * G):
                    z = _wide(st["q"][t:t + m, x]) @ k.t() / math.sqrt(D)
                    z[hidden] = -math.inf
                    z -= torch.logsumexp(z, 1, keepdim=True)
                    out[t:t + m, x] = z.exp_() @ v
    return out


def _exact_pools(case, st, pairs):
    out = []
    for name in ("k", "v", "bounds"):
        x = _wide(st[name])
        before = x.clone()
        for s, d in pairs:
            x[d] = before[s]
        out.append(x)
    return out


def _exact_fork(case, st):
    """One pair after the other, as the definition reads."""
    bs = case["block"]
    table, cached = st["table"].tolist(), st["cached"].tolist()
    stack, top = st["free"].tolist(), int(st["count"])
    shares = st["shares"].tolist()
    seq, src, dst, wanted, used = list(cached), [], [], 0, 0
    rows = zip(st["parents"].tolist(), st["children"].tolist(), st["take"].tolist())
    for p, c, n in rows:
        n = min(max(n, 0), cached[p])
        src.append(-1)
        dst.append(-1)
        if n % bs:
            wanted += 1
            if wanted > top:
                continue
            used = wanted
            dst[-1], src[-1] = stack[top - wanted], table[p][n // bs]
            table[c][n // bs] = dst[-1]
        for j in range(n // bs):
            table[c][j] = table[p][j]
            shares[table[p][j]] += 1
        seq[c] = n
    pairs = [(s, d) for s, d in zip(src, dst) if d >= 0]
    return [_ints(table), _ints(seq), _ints(src), _ints(dst), _ints([top - used]),
            _ints(shares)] + _exact_pools(case, st, pairs)


def _exact_free(case, st):
    bs = case["block"]
    table, cached, keep = st["table"].tolist(), st["cached"].tolist(), st["keep"].tolist()
    held, stack, top = st["shares"].tolist(), st["free"].tolist(), int(st["count"])
    shares, freed, seq = list(held), [], []
    for b, n in enumerate(cached):
        m = min(max(keep[b], 0), n)
        if m < n and m % bs and held[table[b][m // bs]] > 0:
            m = n
        seq.append(m)
        for j in range(-(-m // bs), -(-n // bs)):
            page = table[b][j]
            if shares[page] == 0:
                freed.append(page)
            else:
                shares[page] -= 1
    for page in sorted(freed, reverse=True):
        stack[top] = page
        top += 1
    return [_ints(seq), _ints([top]), _ints(stack), _ints(shares)]


def _exact_compact(case, st):
    bs, nb = case["block"], st["shares"].numel()
    table, cached, shares = st["table"].tolist(), st["cached"].tolist(), st["shares"].tolist()
    stack = st["free"].tolist()
    gone = set(stack[:int(st["count"])])
    remap = [-1 if i in gone else i for i in range(nb)]
    edge = max(case["limit"], nb - len(gone))
    high = [i for i in range(edge, nb) if i not in gone]
    low = [i for i in range(edge) if i in gone]
    pairs = list(zip(high, low))
    for s, d in pairs:
        remap[s] = d
        shares[d], shares[s] = shares[s], 0
    for b, n in enumerate(cached):
        for j in range(-(-n // bs)):
            table[b][j] = remap[table[b][j]]
    now = {r for r in remap if r >= 0}
    left = [i for i in range(nb - 1, -1, -1) if i not in now]
    stack[:len(left)] = left
    pad = [-1] * (nb // 2 - len(pairs))
    return [_ints(table), _ints(stack), _ints([len(left)]), _ints(shares), _ints(remap),
            _ints([s for s, _ in pairs] + pad), _ints([d for _, d in pairs] + pad),
            _ints([len(pairs)])] + _exact_pools(case, st, pairs)


# ---- what a pass cannot do without -------------------------------------------------

def work(case):
    bs = case["block"]
    if case["op"] == "free":
        lens, keep, of = _free_plan(case)
        gone = sum(_blocks(n, bs) - _blocks(m, bs) for n, m in zip(lens, keep))
        # The entries that go, their share counts read and written, ids pushed.
        return dict(bytes=16 * gone + 12 * len(lens) + 8, flops=4 * gone)
    H, D = case["kv_heads"], case["head_dim"]
    e = 1 if case["dtype"] == "fp8" else 2
    block = bs * H * D * e * 2 + H * D * 4  # keys, values and bounds
    if case["op"] == "fork":
        lens, parent, take = _fork_plan(case)
        shared = sum(n // bs for n in take)
        copies = max(0, sum(1 for n in take if n % bs) - case["short_of"])
        return dict(bytes=16 * shared + 2 * copies * block + 24 * len(take)
                    + 8 * (case["parents"] + case["children"]), flops=2 * shared)
    if case["op"] == "compact":
        lens = _spread(case["requests"], case["shortest"], case["longest"])
        lens[0] = case["longest"]
        need = [_blocks(n, bs) for n in lens]
        used = sum(need)
        pool = used + case["holes"]
        again = sum(min(lens[0], lens[b]) * 3 // 4 // bs
                    for b in range(max(1, len(lens) - case["shared"]), len(lens)))
        live = used - again
        edge = min(pool, max(case["limit"], live))
        # Blocks lie at random: a live one is above the edge as often as any.
        moves = int(round((pool - edge) * live / pool))
        return dict(bytes=8 * used + 4 * (pool - live) * 2 + 12 * pool + 2 * moves * block,
                    flops=4 * pool)
    cached, new, total = _chunks(case)
    w, Hq = case["window"], case["heads"]
    keys = pairs = rows = table = 0
    for c, m, n in zip(cached, new, total):
        if n < c + m:
            continue
        rows += m
        lo = max(0, c + 1 - w) if w else 0
        keys += n - lo
        table += _blocks(n, bs) - lo // bs
        # Row i sees min(c + i + 1, w) keys.
        full = min(m, max(0, w - c)) if w else m  # rows before the window cuts
        pairs += full * c + full * (full + 1) // 2 + (m - full) * w
    return dict(bytes=keys * H * D * 2 * e + (rows + sum(new)) * Hq * D * 2 + 4 * table
                + 12 * len(new), flops=4 * pairs * Hq * D)
