"""Cases of the paged key-value cache's operators, for measurement.

One decode step of a served model runs these operators around the value
projection: ``paged_plan`` hands out cache blocks and slots for the step's
tokens, ``kv_store_paged`` writes their keys (and values) and the blocks' key
bounds, ``block_select`` picks the blocks worth reading, and
``attention_paged`` attends one new token per request over the cache, the
whole of it or the picked blocks.

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
        # One user's request right after a short prompt: all latency.
        dict(name="attend_one_short", op="attend", dtype="bf16", batch=1, heads=32, kv_heads=8,
             head_dim=128, block=16, shortest=130, longest=130, window=0, empty=False),
        # The serving batch of the decode benchmark (64 requests), mixed ages.
        dict(name="attend_batch", op="attend", dtype="bf16", batch=64, heads=32, kv_heads=8,
             head_dim=128, block=16, shortest=500, longest=8000, window=0, empty=False),
        # One request at the model's full context of 524,288 tokens.
        dict(name="attend_long", op="attend", dtype="bf16", batch=1, heads=32, kv_heads=8,
             head_dim=128, block=64, shortest=524288, longest=524288, window=0, empty=False),
        # The serving batch with the cache held in 8 bits.
        dict(name="attend_batch_fp8", op="attend", dtype="fp8", batch=64, heads=32, kv_heads=8,
             head_dim=128, block=32, shortest=1000, longest=16000, window=0, empty=False),
        # Another layer shape: narrow heads, a group of 5, a block size that is
        # no power of two, a sliding window and a padded batch row.
        dict(name="attend_odd", op="attend", dtype="bf16", batch=37, heads=15, kv_heads=3,
             head_dim=64, block=24, shortest=3, longest=6001, window=2500, empty=True),
        # Few requests with very long contexts, 64 blocks of 32 tokens read.
        dict(name="sparse_long", op="sparse", dtype="bf16", batch=3, heads=32, kv_heads=8,
             head_dim=128, block=32, shortest=100000, longest=400000, keep=64, first=1, last=2,
             empty=False),
        # A serving batch over an 8-bit cache, 64 blocks of 16 tokens read.
        dict(name="sparse_batch_fp8", op="sparse", dtype="fp8", batch=32, heads=32, kv_heads=8,
             head_dim=128, block=16, shortest=600, longest=30000, keep=64, first=1, last=4,
             empty=True),
        # The keys of one decode step: one new token in each of 64 requests.
        dict(name="store_step", op="store", dtype="bf16", requests=64, tokens=64, kv_heads=8,
             head_dim=128, block=16, values=False, padding=0),
        # Keys and values of a prefill chunk of several prompts, to 8 bits.
        dict(name="store_prompts_fp8", op="store", dtype="fp8", requests=7, tokens=8192,
             kv_heads=8, head_dim=128, block=32, values=True, padding=61),
        # The blocks and slots of one decode step, a few requests ending.
        dict(name="plan_step", op="plan", requests=64, tokens=64, block=16, max_blocks=512,
             ending=3, short_of=0),
        # Prompts and running requests mixed, the pool too small for all.
        dict(name="plan_prompts", op="plan", requests=203, tokens=32768, block=16,
             max_blocks=2048, ending=11, short_of=150),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "sparse", "sparse", "store", "store", "plan"])
    dtype = rng.choice(["bf16", "bf16", "fp8"])
    kv_heads = rng.choice([1, 2, 3, 4, 6, 8, 8])
    group = rng.choice([1, 2, 3, 4, 4, 5, 8, 16])
    head_dim = rng.choice([64, 128, 128, 128, 256])
    block = rng.choice([8, 16, 16, 24, 32, 48, 64, 128])
    if op == "attend":
        batch = _log(rng, 1, 200)
        # Keys read, and products made, stay below the longest listed case's.
        most = min(524288, 500000 * 1024 // (batch * kv_heads * head_dim * max(1, -(-group // 4))))
        longest = _log(rng, 1, most)
        return dict(op=op, dtype=dtype, batch=batch, heads=kv_heads * group, kv_heads=kv_heads,
                    head_dim=head_dim, block=block, shortest=_log(rng, 1, longest),
                    longest=longest, window=rng.choice([0, 0, 0, _log(rng, 1, longest)]),
                    empty=rng.random() < 0.3)
    if op == "sparse":
        batch = _log(rng, 1, 100)
        blocks = 22000 * 1024 // (batch * kv_heads * head_dim * max(1, -(-group // 4)))
        longest = _log(rng, 40, max(40, min(400000, blocks * block)))
        keep = _log(rng, 4, 128)
        last = rng.randint(1, 2)
        return dict(op=op, dtype=dtype, batch=batch, heads=kv_heads * group, kv_heads=kv_heads,
                    head_dim=head_dim, block=block, shortest=_log(rng, 1, longest),
                    longest=longest, keep=keep, first=rng.randint(0, 2), last=last,
                    empty=rng.random() < 0.3)
    if op == "store":
        requests = _log(rng, 1, 200)
        return dict(op=op, dtype=dtype, requests=requests,
                    tokens=requests + _log(rng, 1, 12000) - 1, kv_heads=kv_heads,
                    head_dim=head_dim, block=block, values=rng.random() < 0.5,
                    padding=rng.choice([0, rng.randint(1, 63)]))
    requests = _log(rng, 1, 300)
    tokens = requests + _log(rng, 1, 30000) - 1
    return dict(op=op, requests=requests, tokens=tokens, block=block,
                max_blocks=_log(rng, tokens // block + 600, 20000), ending=rng.randint(0, requests // 4),
                short_of=rng.choice([0, 0, _log(rng, 1, 200)]))


# ---- lengths, the same for every seed -----------------------------------------

def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], even in their logarithm, in mixed order."""
    out = []
    for i in range(n):
        u = (0.31 + i * 0.6180339887498949) % 1.0
        out.append(min(hi, max(lo, int(round(lo * (hi / lo) ** u)))))
    return out


def _lens(case):
    lens = _spread(case["batch"], case["shortest"], case["longest"])
    lens[0] = case["longest"]
    if case["empty"] and len(lens) > 1:
        lens[len(lens) // 2] = 0  # a padded row of the batch
    return lens


def _shares(total, n):
    """total split into n shares of at least one, uneven."""
    w = [x - 1 for x in _spread(n, 2, 400)]
    s = sum(w)
    free = total - n
    out = [1 + free * x // s for x in w]
    out[-1] += total - sum(out)
    return out


def _blocks(n, block):
    return (n + block - 1) // block


def _store_plan(case):
    """Per request: tokens already stored, and new ones."""
    new = _shares(case["tokens"], case["requests"])
    return [(37 * i + 5) % (4 * case["block"]) for i in range(case["requests"])], new


def _plan_lens(case):
    """Stored and new tokens per request (new < 0: the request has ended)."""
    n = case["requests"]
    going = n - case["ending"]
    new = _shares(case["tokens"], going)
    step = n / max(case["ending"], 1)
    ends = {int(i * step) for i in range(case["ending"])}
    cached = _spread(n, 1, 500 * case["block"])
    out, it = [], iter(new)
    for i in range(n):
        out.append(-1 if i in ends else next(it))
        if not i % 5:
            cached[i] = 0 if out[i] > 0 else cached[i]
    return cached, out


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _scales(g, n):
    return (1.0 + torch.rand(n, generator=g, device=DEV)) / 64.0


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


def _tables(g, lens, block, spare, width=None):
    """A random block table for the lengths; entries past a request are -1."""
    need = [_blocks(n, block) for n in lens]
    pool = sum(need) + spare
    perm = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), width or max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pool, perm[at:]


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] in ("attend", "sparse"):
        H, D, bs = case["kv_heads"], case["head_dim"], case["block"]
        lens = _lens(case)
        st["lens"] = lens
        st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st["table"], pool, _ = _tables(g, lens, bs, 3)
        st["q"] = _rows(g, case["batch"], case["heads"], D).to(torch.bfloat16)
        st["k_scale"] = st["v_scale"] = None
        if case["dtype"] == "fp8":
            st["k_scale"], st["v_scale"] = _scales(g, H), _scales(g, H)
        st["k"] = _pool(g, pool, bs, H, D, case["dtype"], st["k_scale"], 1.0)
        st["v"] = _pool(g, pool, bs, H, D, case["dtype"], st["v_scale"], 0.0)
        if case["op"] == "sparse":
            # As the key store leaves them: over the rows that hold keys.
            st["bounds"] = torch.empty(pool, H, 2, D, dtype=torch.bfloat16, device=DEV)
            step = max(1, (1 << 26) // (bs * H * D))
            for i in range(0, pool, step):
                r = st["k"][i:i + step].float()
                st["bounds"][i:i + step, :, 0] = r.amin(1).to(torch.bfloat16)
                st["bounds"][i:i + step, :, 1] = r.amax(1).to(torch.bfloat16)
            for b, n in enumerate(lens):
                if n % bs:
                    p = int(st["table"][b, n // bs])
                    r = st["k"][p, :n % bs].float()
                    st["bounds"][p, :, 0] = r.amin(0).to(torch.bfloat16)
                    st["bounds"][p, :, 1] = r.amax(0).to(torch.bfloat16)
    elif case["op"] == "store":
        H, D, bs = case["kv_heads"], case["head_dim"], case["block"]
        cached, new = _store_plan(case)
        table, pool, _ = _tables(g, [c + n for c, n in zip(cached, new)], bs, 3)
        rows = case["tokens"] + case["padding"]
        slots = torch.full((rows,), -1, dtype=torch.int64, device=DEV)
        at = 0
        for b in range(case["requests"]):
            pos = torch.arange(cached[b], cached[b] + new[b], device=DEV)
            slots[at:at + new[b]] = table[b, pos // bs].long() * bs + pos % bs
            at += new[b]
        st["slots"] = slots
        # What a host-side plan knows beside the slots: the blocks touched,
        # and how many of their rows hold keys after the call.
        touched, filled = [], []
        for b in range(case["requests"]):
            j = torch.arange(cached[b] // bs, _blocks(cached[b] + new[b], bs), device=DEV)
            touched.append(table[b, j].long())
            filled.append((cached[b] + new[b] - j * bs).clamp(max=bs))
        st["touched"], st["filled"] = torch.cat(touched), torch.cat(filled)
        st["k_scale"] = st["v_scale"] = None
        if case["dtype"] == "fp8":
            st["k_scale"], st["v_scale"] = _scales(g, H), _scales(g, H)
        st["new_k"] = _rows(g, rows, H, D).to(torch.bfloat16)
        st["new_v"] = _rows(g, rows, H, D).to(torch.bfloat16) if case["values"] else None
        st["k"] = _pool(g, pool, bs, H, D, case["dtype"], st["k_scale"], 1.0)
        st["v"] = (_pool(g, pool, bs, H, D, case["dtype"], st["v_scale"], 0.0)
                   if case["values"] else None)
        st["bounds"] = torch.zeros(pool, H, 2, D, dtype=torch.bfloat16, device=DEV)
    else:
        bs = case["block"]
        cached, new = _plan_lens(case)
        grow = sum(_blocks(c + n, bs) - _blocks(c, bs) for c, n in zip(cached, new) if n > 0)
        ends = sum(_blocks(c, bs) for c, n in zip(cached, new) if n < 0)
        spare = max(0, grow - ends - case["short_of"]) + (0 if case["short_of"] else 40)
        st["table"], pool, left = _tables(g, cached, bs, spare, case["max_blocks"])
        st["free"] = torch.full((pool,), -1, dtype=torch.int32, device=DEV)
        st["free"][:left.numel()] = left
        st["count"] = torch.tensor([left.numel()], dtype=torch.int32, device=DEV)
        st["cached"] = torch.tensor(cached, dtype=torch.int32, device=DEV)
        st["new"] = torch.tensor(new, dtype=torch.int32, device=DEV)
    return st


# ---- one pass -----------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return {"attend": _own_attend, "sparse": _own_sparse, "store": _own_store,
                "plan": _own_plan}[op](st)
    return {"attend": _attend, "sparse": _sparse, "store": _store, "plan": _plan}[op](st)


def _own_attend(st):
    from mixture_value_projection_amd import binding
    case = st["case"]
    return binding.attention_paged(st["q"], st["k"], st["v"], st["table"], st["seq_lens"],
                                   case["head_dim"] ** -0.5, k_scale=st["k_scale"],
                                   v_scale=st["v_scale"], window=case["window"])


def _own_sparse(st):
    from mixture_value_projection_amd import binding
    case = st["case"]
    sel = binding.block_select(st["q"], st["bounds"], case["block"], st["table"], st["seq_lens"],
                               case["keep"], keep_first=case["first"], keep_last=case["last"])
    out = binding.attention_paged(st["q"], st["k"], st["v"], st["table"], st["seq_lens"],
                                  case["head_dim"] ** -0.5, k_scale=st["k_scale"],
                                  v_scale=st["v_scale"], sel_blocks=sel)
    return sel, out


def _own_store(st):
    from mixture_value_projection_amd import binding
    binding.kv_store_paged(st["new_k"], st["new_v"], st["k"], st["v"], st["slots"],
                           k_scale=st["k_scale"], v_scale=st["v_scale"], k_bounds=st["bounds"])
    return [t for t in (st["k"], st["v"], st["bounds"]) if t is not None]


def _own_plan(st):
    from mixture_value_projection_amd import binding
    case = st["case"]
    p = binding.paged_plan(st["cached"], st["new"], case["tokens"], case["block"], st["table"],
                           st["free"], st["count"])
    return [st["table"], st["free"], p.seq_lens, p.cu_new, p.slot_mapping, p.positions,
            p.free_count]


# ---- the plain forms ------------------------------------------------------------

def _softmax_rows(q, k, v, scale, v_scale):
    """One request: q [H, G, D], k and v [H, n, D], all float32."""
    s = torch.matmul(q, k.transpose(1, 2)) * scale
    s = s - s.amax(-1, keepdim=True)
    p = torch.exp(s)
    o = torch.matmul(p / p.sum(-1, keepdim=True), v)
    return o if v_scale is None else o * v_scale[:, None, None]


def _logit_scale(case, k_scale):
    s = case["head_dim"] ** -0.5
    return s if k_scale is None else (k_scale * s)[:, None, None]


def _attend(st):
    case = st["case"]
    H, D, bs = case["kv_heads"], case["head_dim"], case["block"]
    G = case["heads"] // H
    out = torch.zeros(case["batch"], case["heads"], D, device=DEV)
    scale = _logit_scale(case, st["k_scale"])
    for b, n in enumerate(st["lens"]):
        if n == 0:
            continue
        lo = max(0, n - case["window"]) if case["window"] else 0
        j0 = lo // bs
        ids = st["table"][b, j0:_blocks(n, bs)].long()
        k = st["k"][ids].reshape(-1, H, D)[lo - j0 * bs:n - j0 * bs].float().transpose(0, 1)
        v = st["v"][ids].reshape(-1, H, D)[lo - j0 * bs:n - j0 * bs].float().transpose(0, 1)
        q = st["q"][b].float().reshape(H, G, D)
        out[b] = _softmax_rows(q, k.contiguous(), v.contiguous(), scale,
                               st["v_scale"]).reshape(case["heads"], D)
    return out.to(torch.bfloat16)


def _sparse(st):
    case = st["case"]
    H, D, bs, keep = case["kv_heads"], case["head_dim"], case["block"], case["keep"]
    G = case["heads"] // H
    out = torch.zeros(case["batch"], case["heads"], D, device=DEV)
    sel = torch.full((case["batch"], H, keep), -1, dtype=torch.int32, device=DEV)
    scale = _logit_scale(case, st["k_scale"])
    heads = torch.arange(H, device=DEV)[:, None]
    for b, n in enumerate(st["lens"]):
        if n == 0:
            continue
        nb = _blocks(n, bs)
        ids = st["table"][b, :nb].long()
        q = st["q"][b].float().reshape(H, G, D)
        # The largest a key of the block can make q . k, in 64 bits: the
        # choice between two blocks is as fine as their difference.
        lo, hi = st["bounds"][ids, :, 0].double(), st["bounds"][ids, :, 1].double()  # [nb, H, D]
        score = torch.full((nb, H), -math.inf, dtype=torch.float64, device=DEV)
        for g in range(G):
            qg = q[:, g].double()
            score = torch.maximum(score, (torch.where(qg > 0, hi, lo) * qg).sum(-1))
        score[:case["first"]] = math.inf
        score[max(0, nb - case["last"]):] = math.inf
        rank = torch.sort(score.t().contiguous(), dim=1, descending=True, stable=True).indices
        pick = torch.sort(rank[:, :keep], dim=1).values  # [H, kept]
        sel[b, :, :pick.shape[1]] = pick.to(torch.int32)
        phys = ids[pick]
        k = st["k"][phys, :, heads].float().reshape(H, -1, D)
        v = st["v"][phys, :, heads].float().reshape(H, -1, D)
        # The last block is always picked and last in the list: the rows past
        # the length are the list's end, the same number for every head.
        m = int(pick.shape[1]) * bs - (nb * bs - n)
        out[b] = _softmax_rows(q, k[:, :m].contiguous(), v[:, :m].contiguous(), scale,
                               st["v_scale"]).reshape(case["heads"], D)
    return sel, out.to(torch.bfloat16)


def _store(st):
    case = st["case"]
    bs, n = case["block"], case["tokens"]
    H, D = case["kv_heads"], case["head_dim"]
    slots = st["slots"][:n]
    for new, pool, scale in ((st["new_k"], st["k"], st["k_scale"]),
                             (st["new_v"], st["v"], st["v_scale"])):
        if new is None:
            continue
        x = new[:n]
        if case["dtype"] == "fp8":
            x = (x.float() / scale[:, None]).clamp(-FP8_MAX, FP8_MAX).to(FP8)
            pool.view(torch.uint8).view(-1, H, D)[slots] = x.view(torch.uint8)
        else:
            pool.view(-1, H, D)[slots] = x
    rows = st["k"].view(torch.uint8)[st["touched"]].view(FP8) if case["dtype"] == "fp8" \
        else st["k"][st["touched"]]
    rows = rows.float()
    held = (torch.arange(bs, device=DEV) < st["filled"][:, None])[:, :, None, None]
    st["bounds"][st["touched"], :, 0] = torch.where(held, rows, math.inf).amin(1).to(torch.bfloat16)
    st["bounds"][st["touched"], :, 1] = torch.where(held, rows, -math.inf).amax(1).to(torch.bfloat16)
    return [t for t in (st["k"], st["v"], st["bounds"]) if t is not None]


def _plan(st):
    case = st["case"]
    bs, T, mb = case["block"], case["tokens"], case["max_blocks"]
    cached, new, table, free = st["cached"].long(), st["new"].long(), st["table"], st["free"]
    count = st["count"].long()
    ended = new < 0
    tok = new.clamp(min=0)
    cu = torch.cat([tok.new_zeros(1), tok.cumsum(0)])
    old = (cached + bs - 1) // bs
    total = cached + tok
    fits = ~ended & (total <= mb * bs) & (cu[1:] <= T)
    need = torch.where(fits, (total + bs - 1) // bs - old, 0)
    back = torch.where(ended, old, 0)
    col = torch.arange(mb, device=DEV)
    ids = table[col < back[:, None]]
    free[count + torch.arange(ids.numel(), device=DEV)] = ids
    have = count + ids.numel()
    upto = need.cumsum(0)
    ok = fits & ((need == 0) | (upto <= have))
    taken = torch.where(ok & (need > 0), upto, 0).amax()
    new_blocks = (col >= old[:, None]) & (col < (old + need)[:, None]) & ok[:, None]
    order = torch.arange(int(taken), device=DEV)
    table[new_blocks] = free[have - 1 - order]
    seq = torch.where(ended, 0, torch.where(ok, total, cached))
    slots = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    where = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    req = torch.repeat_interleave(torch.arange(cached.numel(), device=DEV), tok)[:T]
    pos = cached[req] + torch.arange(req.numel(), device=DEV) - cu[req]
    page = table[req, (pos // bs).clamp(max=mb - 1)].long()
    slots[:req.numel()] = torch.where(ok[req], page * bs + pos % bs, -1)
    where[:req.numel()] = torch.where(ok[req], pos, -1).to(torch.int32)
    return [table, free, seq.to(torch.int32), cu.to(torch.int32), slots, where,
            (have - taken).to(torch.int32)]


# ---- the definitions in 64 bits ---------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"attend": _exact_attend, "sparse": _exact_sparse, "store": _exact_store,
            "plan": _exact_plan}[case["op"]](case, st)


def _wide(t):
    return t.float().double()


def _exact_row(q, k, v, scale):
    """One query head: q [D], k and v [n, D] in float64."""
    z = (k * q).sum(1) * scale
    w = torch.exp(z - torch.logsumexp(z, 0))
    return (w[:, None] * v).sum(0)


def _exact_keys(case, st, b, positions):
    """Float64 keys and values [n, H, D] of request b at the positions."""
    bs = case["block"]
    page, off = st["table"][b].long()[positions // bs], positions % bs
    k, v = _wide(st["k"][page, off]), _wide(st["v"][page, off])
    if st["k_scale"] is not None:
        k = k * _wide(st["k_scale"])[:, None]
        v = v * _wide(st["v_scale"])[:, None]
    return k, v


def _exact_attend(case, st):
    G = case["heads"] // case["kv_heads"]
    out = torch.zeros(case["batch"], case["heads"], case["head_dim"], dtype=torch.float64,
                      device=DEV)
    for b, n in enumerate(_lens(case)):
        start = n - case["window"] if 0 < case["window"] < n else 0
        if n == 0:
            continue
        k, v = _exact_keys(case, st, b, torch.arange(start, n, device=DEV))
        for h in range(case["heads"]):
            out[b, h] = _exact_row(_wide(st["q"][b, h]), k[:, h // G], v[:, h // G],
                                   1.0 / math.sqrt(case["head_dim"]))
    return out


def _exact_sparse(case, st):
    G, bs = case["heads"] // case["kv_heads"], case["block"]
    H = case["kv_heads"]
    out = torch.zeros(case["batch"], case["heads"], case["head_dim"], dtype=torch.float64,
                      device=DEV)
    sel = torch.full((case["batch"], H, case["keep"]), -1, dtype=torch.int32, device=DEV)
    for b, n in enumerate(_lens(case)):
        if n == 0:
            continue
        nb = -(-n // bs)
        box = _wide(st["bounds"][st["table"][b, :nb].long()])  # [nb, H, 2, D]
        for h in range(H):
            best = None
            for g in range(G):
                q = _wide(st["q"][b, h * G + g])
                s = torch.maximum(box[:, h, 0] * q, box[:, h, 1] * q).sum(1)
                best = s if best is None else torch.maximum(best, s)
            best = best.tolist()
            forced = [j for j in range(nb) if j < case["first"] or j >= nb - case["last"]]
            rest = sorted(set(range(nb)) - set(forced), key=lambda j: (-best[j], j))
            got = sorted((forced + rest)[:case["keep"]])
            sel[b, h, :len(got)] = torch.tensor(got, dtype=torch.int32, device=DEV)
            pos = torch.tensor(got, device=DEV)[:, None] * bs + torch.arange(bs, device=DEV)
            pos = pos.reshape(-1)
            k, v = _exact_keys(case, st, b, pos[pos < n])
            for g in range(G):
                out[b, h * G + g] = _exact_row(_wide(st["q"][b, h * G + g]), k[:, h], v[:, h],
                                               1.0 / math.sqrt(case["head_dim"]))
    return sel, out


def _exact_store(case, st):
    H, D, bs = case["kv_heads"], case["head_dim"], case["block"]
    out = []
    for new, pool, scale in ((st["new_k"], st["k"], st["k_scale"]),
                             (st["new_v"], st["v"], st["v_scale"])):
        if new is None:
            continue
        rows = _wide(pool).reshape(-1, H, D)
        x = _wide(new)
        if scale is not None:
            x = torch.clamp(x / _wide(scale)[None, :, None], -FP8_MAX, FP8_MAX)
        held = st["slots"] >= 0
        rows[st["slots"][held]] = x[held]
        out.append(rows.reshape(pool.shape))
    # The bounds are those of the rows as the pool holds them: with an 8-bit
    # pool, of rounded values.
    keys = out[0].clone().reshape(-1, H, D)
    if case["dtype"] == "fp8":
        keys = _wide(keys.float().to(FP8))
    keys = keys.reshape(-1, bs, H, D)
    bounds = torch.zeros(keys.shape[0], H, 2, D, dtype=torch.float64, device=DEV)
    for p, n in zip(st["touched"].tolist(), st["filled"].tolist()):
        bounds[p, :, 0] = keys[p, :n].min(0).values
        bounds[p, :, 1] = keys[p, :n].max(0).values
    return out + [bounds]


def _exact_plan(case, st):
    """One request after the other, as the definition reads."""
    bs, T, mb = case["block"], case["tokens"], case["max_blocks"]
    cached, new = st["cached"].tolist(), st["new"].tolist()
    table, stack = st["table"].tolist(), st["free"].tolist()
    top = int(st["count"])
    for b, n in enumerate(new):
        if n < 0:
            for j in range(-(-cached[b] // bs)):
                stack[top] = table[b][j]
                top += 1
    have, wanted, used = top, 0, 0
    seq, cu, slots, where = [], [0], [-1] * T, [-1] * T
    for b, n in enumerate(new):
        m = max(n, 0)
        cu.append(cu[-1] + m)
        if n < 0:
            seq.append(0)
            continue
        size = cached[b] + m
        seq.append(cached[b])
        if size > mb * bs or cu[-1] > T:
            continue
        have_now = -(-cached[b] // bs)
        more = -(-size // bs) - have_now
        wanted += more
        if more and wanted > have:
            continue
        for j in range(more):
            table[b][have_now + j] = stack[have - 1 - (wanted - more) - j]
        used = max(used, wanted if more else 0)
        seq[b] = size
        for i in range(m):
            p = cached[b] + i
            slots[cu[b] + i] = table[b][p // bs] * bs + p % bs
            where[cu[b] + i] = p

    def ints(x, t=torch.int32):
        return torch.tensor(x, dtype=t, device=DEV)
    return [ints(table), ints(stack), ints(seq), ints(cu), ints(slots, torch.int64), ints(where),
            ints([have - used])]


# ---- what a pass cannot do without -------------------------------------------------

def work(case):
    if case["op"] == "plan":
        cached, new = _plan_lens(case)
        bs, T, B = case["block"], case["tokens"], case["requests"]
        back = sum(_blocks(c, bs) for c, n in zip(cached, new) if n < 0)
        more = sum(_blocks(c + n, bs) - _blocks(c, bs) for c, n in zip(cached, new) if n > 0)
        more = max(0, more - case["short_of"])
        return dict(bytes=8 * B + 8 * (back + more) + 8 * B + 8 + 12 * T, flops=4 * T)
    H, D = case["kv_heads"], case["head_dim"]
    e = 1 if case["dtype"] == "fp8" else 2
    if case["op"] == "store":
        cached, new = _store_plan(case)
        bs = case["block"]
        sides = 2 if case["values"] else 1
        touched = sum(_blocks(c + n, bs) - c // bs for c, n in zip(cached, new))
        before = sum(c % bs for c in cached)
        T = case["tokens"]
        return dict(bytes=sides * T * H * D * (2 + e) + before * H * D * e + touched * H * D * 4
                    + 8 * (T + case["padding"]),
                    flops=(2 * (T + before) + sides * T * (2 if e == 1 else 0)) * H * D)
    lens, bs, Hq, B = _lens(case), case["block"], case["heads"], case["batch"]
    small = B * Hq * D * 4 + 4 * B + 4 * sum(_blocks(n, bs) for n in lens)
    if case["op"] == "attend":
        w = case["window"]
        keys = sum(min(n, w) if w else n for n in lens)
        return dict(bytes=keys * H * D * 2 * e + small, flops=4 * keys * Hq * D)
    blocks = sum(_blocks(n, bs) for n in lens)
    keys = sum(min(n, case["keep"] * bs - (-n) % bs) for n in lens)
    return dict(bytes=blocks * H * D * 4 + keys * H * D * 2 * e + small
                + 4 * B * H * case["keep"],
                flops=2 * blocks * Hq * D + 4 * keys * Hq * D)
