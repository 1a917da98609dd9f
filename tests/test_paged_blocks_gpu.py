"""Upkeep of the paged cache's blocks (fork, free, compaction, copy) against
plain references, and a run of it around the attention."""
import numpy as np
import pytest
import torch

from mixture_value_projection_amd import binding
import blockslib as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
FP8 = R.FP8
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu_only():
    assert torch.cuda.is_available(), "GPU test run without a GPU"
    binding.load_library()


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device=DEV)


def host(*tensors):
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in tensors]


def same(got, want, names, what):
    for g, w, n in zip(got, want, names):
        w = np.asarray(w)
        assert np.array_equal(np.asarray(g).reshape(w.shape), w), f"{what}: {n}"


def state(seed, B, bs, mb, longest, spare, empty=0, share=0):
    """A pool with B rows of random lengths, the last `empty` without tokens,
    `share` rows sharing part of row 0: (lens, table, free, count, shares)."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, B)
    lens[0] = longest
    if empty:
        lens[-empty:] = 0
    need = [R.ceil_div(int(n), bs) for n in lens]
    nb = sum(need) + spare
    perm = rng.permutation(nb)
    table = np.full((B, mb), -1)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    left, shares = list(perm[at:]), np.zeros(nb, dtype=np.int64)
    for b in range(1, 1 + share):
        c = int(rng.integers(0, min(lens[0], lens[b]) // bs + 1))
        left += list(table[b, :c])
        table[b, :c] = table[0, :c]
        shares[table[0, :c]] += 1
    free = np.full(nb, -1)
    free[:len(left)] = left
    return lens, table, free, len(left), shares


# ---- fork -----------------------------------------------------------------------

FORK = ("table", "seq_lens", "copy_src", "copy_dst", "free_count", "shares")


def check_fork(parents, children, take, lens, bs, table, free, count, shares, what):
    want = R.fork(parents, children, take, lens, bs, table, free, count, shares)
    t, f, s = i32(table), i32(free), i32(shares)
    p = binding.paged_fork(i32(parents), i32(children), bs, t, i32(lens), f, i32([count]), s,
                           fork_lens=None if take is None else i32(take))
    got = host(t, p.seq_lens, p.copy_src, p.copy_dst, p.free_count, s)
    same(got, want, FORK, what)
    assert np.array_equal(host(f)[0], free), f"{what}: the stack"


@pytest.mark.parametrize("seed,B,n,bs,longest,spare", [
    (0, 2, 1, 16, 0, 3), (1, 2, 1, 16, 40, 3), (2, 40, 30, 16, 900, 50), (3, 40, 30, 24, 900, 5),
    (4, 300, 200, 8, 600, 90), (5, 2048, 1800, 16, 60, 2000), (6, 9, 8, 1, 300, 0),
    (7, 12, 11, 128, 9000, 20), (8, 5, 4, 16, 30000, 9),
])
@pytest.mark.parametrize("prefixes", [False, True])
def test_fork(seed, B, n, bs, longest, spare, prefixes):
    rng = np.random.default_rng(seed)
    # (Rows of the parents alone: the children's are empty.)
    lens, table, free, count, shares = state(seed, B, bs, R.ceil_div(longest, bs) + 3, longest,
                                             spare, empty=n)
    parents = rng.integers(0, B - n, n)
    children = B - n + rng.permutation(n)
    take = None
    if prefixes:
        take = rng.integers(-2, longest + 20, n)
        take[::3] = take[::3] // bs * bs
    check_fork(parents, children, take, lens, bs, table, free, count, shares, "fork")


def test_fork_pairs_that_get_nothing():
    """Rows outside the table, a row forked to itself, a child named twice, a
    child that is a parent, padding, an empty list."""
    lens, table, free, count, shares = state(9, 12, 16, 30, 200, 9, empty=6, share=2)
    args = (lens, 16, table, free, count, shares)
    check_fork([0, 1, -1, 12, 2, 3, 0, 0, 7], [6, 6, 8, 9, -5, 12, 0, 7, 8], None, *args, "nothing")
    check_fork([0, 6, 6], [6, 7, 8], None, *args, "a child that is a parent")
    check_fork([0, 6], [6, 12], None, *args, "a parent of a pair that gets nothing")
    check_fork([0, 1, 2], [6, 6, 6], [5, 40, 32], *args, "a child named three times")
    check_fork([-1] * 5, [-1] * 5, None, *args, "padding")
    check_fork([], [], None, *args, "none")


@pytest.mark.parametrize("count", [0, 1, 2, 3, -4, 1000])
def test_fork_short_of_blocks(count):
    lens, table, free, _, shares = state(10, 12, 16, 30, 200, 9, empty=6)
    lens[:6] = [200, 33, 48, 15, 100, 7]
    check_fork([0, 2, 1, 3, 2, 5], range(6, 12), None, lens, 16, table, free, count, shares,
               f"{count} free")


def test_fork_of_missing_blocks():
    lens, table, free, count, shares = state(11, 8, 16, 30, 200, 9, empty=4)
    nb = len(shares)
    table[0, 1], table[0, 3], table[0, 12] = -1, nb, nb + 5
    check_fork([0, 0, 0], [5, 6, 7], [200, 52, 199], lens, 16, table, free, count, shares, "missing")


# ---- free -----------------------------------------------------------------------

FREE = ("seq_lens", "free_count", "free", "shares")


def check_free(lens, keep, bs, table, free, count, shares, what):
    want = R.release(lens, keep, bs, table, free, count, shares)
    f, s = i32(free), i32(shares)
    p = binding.paged_free(i32(lens), i32(keep), bs, i32(table), f, i32([count]), s)
    same(host(p.seq_lens, p.free_count, f, s), want, FREE, what)


@pytest.mark.parametrize("seed,B,bs,longest,spare,share", [
    (0, 1, 16, 0, 1, 0), (1, 1, 16, 70, 0, 0), (2, 64, 16, 900, 20, 0), (3, 64, 24, 900, 20, 30),
    (4, 300, 8, 600, 50, 299), (5, 2048, 16, 90, 33, 1500), (6, 20, 1, 500, 7, 15),
    (7, 9, 128, 12000, 0, 5), (8, 40, 16, 12000, 64, 39),
])
def test_free(seed, B, bs, longest, spare, share):
    rng = np.random.default_rng(seed)
    lens, table, free, count, shares = state(seed, B, bs, R.ceil_div(longest, bs) + 2, longest,
                                             spare, share=share)
    args = (bs, table, free, count, shares)
    check_free(lens, np.zeros(B), *args, "all end")
    check_free(lens, lens, *args, "none")
    check_free(lens, lens - rng.integers(0, 8, B), *args, "some tokens")
    check_free(lens, np.where(rng.random(B) < 0.4, 0, lens - 3), *args, "mixed")
    check_free(lens, rng.integers(-5, longest + 9, B), *args, "any length")
    check_free(lens, rng.integers(0, longest + 9, B) // bs * bs, *args, "whole blocks")


@pytest.mark.parametrize("nb", [1023, 1025, 131073, 262145, 300001])
def test_free_over_large_pools(nb):
    """Blocks from all over the pool, more than the stack has room for."""
    rng = np.random.default_rng(nb)
    B, mb = 9, 110
    table = rng.permutation(nb)[:B * mb].reshape(B, mb)
    table[0, 0], table[1, 1] = nb - 1, 0
    table[2:, :][(table[2:] == nb - 1) | (table[2:] == 0)] = -1
    shares = np.zeros(nb, dtype=np.int64)
    table[3, :20] = table[2, :20]
    for p in table[3, :20]:
        if p >= 0:
            shares[p] += 1
    lens = np.full(B, mb * 4)
    for keep, cap in ((np.zeros(B), nb), (np.array([0, 9, 400, 0, 3, 0, 0, 8, 440]), nb),
                      (np.zeros(B), 300)):
        free = np.full(cap, -7)
        check_free(lens, keep, 4, table, free, 5, shares, f"{nb} blocks, room for {cap}")


def test_free_last_holder():
    """A block of four holders comes back with the fourth."""
    table = np.array([[3, 1, -1], [3, 2, -1], [3, 0, -1], [3, 4, 5]])
    shares = np.array([0, 0, 0, 3, 0, 0, 0])
    free, lens = np.array([6, -1, -1, -1, -1, -1, -1]), np.array([32, 30, 17, 40])
    for keep in ([0, 0, 0, 40], [0, 0, 0, 0], [16, 16, 16, 16], [0, 16, 0, 16], [5, 30, 17, 40],
                 [8, 8, 8, 8], [0, 0, 0, 7]):
        check_free(lens, keep, 16, table, free, 1, shares, str(keep))


def test_free_onto_a_full_stack_and_missing_blocks():
    lens, table, free, count, shares = state(12, 30, 16, 40, 500, 9, share=10)
    table[0, 2], table[1, 0], table[3, 1] = -1, len(shares), len(shares) + 9
    for cap in (count, count + 5):
        check_free(lens, np.zeros(30), 16, table, free[:cap], count, shares, f"capacity {cap}")
    for c in (-3, 10 ** 6):
        check_free(lens, lens // 2, 16, table, free, c, shares, f"count {c}")
    check_free(lens, np.zeros(30), 16, table, free[:0], 0, shares, "no stack")


@pytest.mark.parametrize("nb", [1, 31, 32, 33, 1024, 32768, 32769, 1 << 20])
def test_free_pool_sizes(nb):
    """Blocks at both ends of the pool's bits."""
    ids = sorted({0, nb - 1, nb // 2, nb // 3, max(nb - 33, 0), min(31, nb - 1), min(32, nb - 1)})
    table = np.array([ids])
    free = np.full(nb, -1)
    check_free([len(ids) * 16], [0], 16, table, free, 0, np.zeros(nb), str(nb))


# ---- compaction -------------------------------------------------------------------

COMPACT = ("table", "free", "free_count", "shares", "remap", "move_src", "move_dst", "move_count")


def check_compact(lens, bs, table, free, count, shares, limit, what):
    want = R.compact(lens, bs, table, free, count, shares, limit)
    t, f, s, c = i32(table), i32(free), i32(shares), i32([count])
    apart = dict(block_table_out=torch.full_like(t, 99), free_blocks_out=torch.full_like(f, 99),
                 shares_out=torch.full_like(s, 99))
    p = binding.paged_compact(i32(lens), bs, t, f, c, s, limit=limit, **apart)
    same(host(*p), want, COMPACT, what + ", apart")
    for g, w in zip(host(t, f, s), (table, free, shares)):
        assert np.array_equal(g, w), what
    p = binding.paged_compact(i32(lens), bs, t, f, c, s, limit=limit)
    assert p.block_table is t and p.free_blocks is f and p.shares is s
    same(host(*p), want, COMPACT, what + ", in place")


@pytest.mark.parametrize("seed,B,bs,longest,spare,share", [
    (0, 1, 16, 0, 1, 0), (1, 1, 16, 70, 0, 0), (2, 64, 16, 900, 400, 0), (3, 64, 24, 900, 20, 30),
    (4, 300, 8, 600, 5000, 299), (5, 2048, 16, 90, 333, 1500), (6, 20, 1, 500, 7, 15),
    (7, 9, 128, 12000, 300, 5), (8, 40, 16, 12000, 64, 39),
])
def test_compact(seed, B, bs, longest, spare, share):
    args = state(seed, B, bs, R.ceil_div(longest, bs) + 2, longest, spare, share=share)
    nb = len(args[4])
    for limit in (0, nb // 2, nb - 1, nb, nb + 100, 2 ** 31 - 1):
        check_compact(args[0], bs, *args[1:], limit, f"limit {limit}")


@pytest.mark.parametrize("nb", [1, 2, 255, 256, 257, 1000, 65536, 1 << 20])
@pytest.mark.parametrize("used", [0, 1, 0.5, 1.0])
def test_compact_pool_sizes(nb, used):
    rng = np.random.default_rng(nb)
    n = int(used * nb) if isinstance(used, float) else min(used, nb)
    perm = rng.permutation(nb)
    table = np.full((3, max(n, 1)), -1)
    table[1, :n] = perm[:n]
    free = np.concatenate([perm[n:], np.full(n, -1)])
    check_compact([0, n, 0], 1, table, free, nb - n, rng.integers(0, 3, nb), 0, f"{n} of {nb}")


def test_compact_odd_stacks():
    """A block on the stack twice, entries outside the pool, counts outside
    the stack, blocks that no row holds, rows that name free blocks."""
    lens, table, free, count, shares = state(13, 20, 16, 40, 500, 90, share=5)
    nb = len(shares)
    free[3], free[5], free[7] = free[2], nb + 3, -9
    check_compact(lens, 16, table, free, count, shares, 0, "odd entries")
    check_compact(lens, 16, table, free, -5, shares, 0, "nothing free")
    check_compact(lens, 16, table, free, 10 ** 6, shares, 0, "all of the stack")
    check_compact(lens, 16, table, free[:10], 10, shares, 0, "short stack")
    table[2, 0], table[4, 1] = nb, -1
    check_compact(lens - 700, 16, table, free, count, shares, 0, "no lengths")
    check_compact(lens + 10 ** 6, 16, table, free, count, shares, 0, "lengths past the row")


# ---- copy -----------------------------------------------------------------------

@pytest.mark.parametrize("H,D,bs,dtype", [(8, 128, 16, BF16), (8, 128, 32, FP8), (1, 16, 1, FP8),
                                          (3, 64, 24, BF16), (1, 256, 1, BF16), (5, 48, 7, FP8)])
@pytest.mark.parametrize("given", ["kvb", "k", "v", "kb", "kv"])
def test_copy(H, D, bs, dtype, given):
    g = torch.Generator().manual_seed(bs)
    nb = 41
    pools = [torch.randint(0, 255, (nb, bs, H, D), generator=g, dtype=torch.uint8).view(FP8)
             if dtype == FP8 else torch.randn(nb, bs, H, D, generator=g).to(BF16) for _ in range(2)]
    pools.append(torch.randn(nb, H, 2, D, generator=g).to(BF16))
    perm = np.random.default_rng(1).permutation(nb)
    src, dst = perm[:20].copy(), perm[20:40].copy()
    src[3], dst[5], src[7], dst[9], dst[11] = -1, -1, nb, nb + 1, src[11]
    for count in (None, 0, 13, 500, -2):
        dev = [p.to(DEV) if x in given else None for p, x in zip(pools, "kvb")]
        binding.paged_copy(i32(src), i32(dst), dev[0], dev[1], k_bounds=dev[2],
                           count=None if count is None else i32([count]))
        torch.cuda.synchronize()
        n = 20 if count is None else min(max(count, 0), 20)
        for p, d in zip(pools, dev):
            if d is None:
                continue
            raw = p.view(torch.uint8) if p.dtype == FP8 else p
            want = raw.clone()
            for s, t in zip(src[:n], dst[:n]):
                if 0 <= s < nb and 0 <= t < nb:
                    want[t] = raw[s]
            got = d.cpu()
            assert torch.equal(got.view(torch.uint8) if p.dtype == FP8 else got, want)


def test_copy_of_many_pairs():
    """More items than workgroups."""
    nb, n = 9000, 4000
    pool = torch.arange(nb * 16 * 64, dtype=torch.int32).view(torch.bfloat16).reshape(nb, 16, 2, 64)
    perm = torch.randperm(nb)
    src, dst = perm[:n], perm[n:2 * n]
    d = pool.to(DEV)
    binding.paged_copy(i32(src.numpy()), i32(dst.numpy()), d, None)
    want = pool.clone().view(torch.int16)
    want[dst] = want[src]
    assert torch.equal(d.cpu().view(torch.int16), want)


# ---- together ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_a_life_of_the_cache(dtype):
    """Prompts stored and attended, forked, the forks' next tokens stored, some
    ended and others cut back, the pool moved together: at every stage the
    attention over the cache is that over the requests' own tokens."""
    g = torch.Generator(device=DEV).manual_seed(3)
    B, mb, bs, H, Hq, D, nb = 10, 24, 16, 2, 8, 64, 80
    k_cache = torch.full((nb, bs, H, D), float("nan"), device=DEV).to(dtype)
    v_cache = k_cache.clone()
    bounds = torch.zeros(nb, H, 2, D, dtype=BF16, device=DEV)
    ks = vs = None
    if dtype == FP8:
        ks, vs = torch.full((H,), 1 / 32, device=DEV), torch.full((H,), 1 / 64, device=DEV)
    table = torch.full((B, mb), -1, dtype=torch.int32, device=DEV)
    free, count = i32(np.random.default_rng(0).permutation(nb)), i32([nb])
    shares = torch.zeros(nb, dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    text = [torch.zeros(0, 2, H, D, dtype=BF16, device=DEV) for _ in range(B)]

    def rows(n):
        return torch.randn(n, H, D, generator=g, device=DEV).to(BF16)

    def own(t, side):
        """The elements that the pool should hold for a request's tokens."""
        x = t[:, side].float()
        if dtype == FP8:
            s = (ks if side == 0 else vs)[:, None]
            x = (x / s).clamp(-448, 448).to(FP8).float() * s
        return x.cpu()

    def attend(cached, p, new):
        q = torch.randn(sum(new), Hq, D, generator=g, device=DEV).to(BF16)
        out = binding.attention_chunk_paged(q, k_cache, v_cache, table, cached, p.seq_lens,
                                            p.cu_new, D ** -0.5, k_scale=ks, v_scale=vs).cpu()
        assert torch.isfinite(out.float()).all()
        at = 0
        for b, n in enumerate(new):
            m = text[b].shape[0]
            k, v = own(text[b], 0).double(), own(text[b], 1).double()
            for i in range(n):
                for h in range(Hq):
                    z = k[:m - n + i + 1, h // 4] @ q[at + i, h].cpu().double() * D ** -0.5
                    want = torch.softmax(z, 0) @ v[:m - n + i + 1, h // 4]
                    off = (out[at + i, h].double() - want).abs().max()
                    # Two roundings to bf16 of numbers below 8.
                    assert off <= 2 * 2.0 ** -8 * 8, (b, i, h)
            at += n

    def step(new):
        nonlocal lens, count
        T = max(sum(new), 1)
        p = binding.paged_plan(lens, i32(new), T, bs, table, free, count)
        assert host(p.seq_lens)[0].tolist() == [t.shape[0] + n for t, n in zip(text, new)]
        k, v = rows(T), rows(T)
        binding.kv_store_paged(k, v, k_cache, v_cache, p.slot_mapping, k_scale=ks, v_scale=vs,
                               k_bounds=bounds)
        at = 0
        for b, n in enumerate(new):
            text[b] = torch.cat([text[b], torch.stack([k[at:at + n], v[at:at + n]], 1)])
            at += n
        attend(lens, p, new)
        lens, count = p.seq_lens, p.free_count

    step([100, 37, 64, 0, 0, 0, 0, 0, 0, 0])
    f = binding.paged_fork(i32([0, 0, 1, 2, 0]), i32([3, 4, 5, 6, 7]), bs, table, lens, free, count,
                           shares, fork_lens=i32([100, 50, 37, 64, 96]))
    binding.paged_copy(f.copy_src, f.copy_dst, k_cache, v_cache, k_bounds=bounds)
    lens, count = f.seq_lens, f.free_count
    for p, c, n in zip([0, 0, 1, 2, 0], [3, 4, 5, 6, 7], [100, 50, 37, 64, 96]):
        text[c] = text[p][:n].clone()
    step([4, 1, 3, 1, 20, 0, 1, 2, 9, 0])
    # Drafts dropped, two requests ended; row 6 is not cut inside a shared block.
    keep = [101, 38, 64, 101, 0, 37, 40, 97, 0, 0]
    r = binding.paged_free(lens, i32(keep), bs, table, free, count, shares)
    lens, count = r.seq_lens, r.free_count
    for b, n in enumerate(keep):
        text[b] = text[b][:65 if b == 6 else n]
    assert host(lens)[0].tolist() == [t.shape[0] for t in text]
    step([1, 1, 1, 2, 0, 1, 1, 1, 5, 0])
    c = binding.paged_compact(lens, bs, table, free, count, shares)
    binding.paged_copy(c.move_src, c.move_dst, k_cache, v_cache, k_bounds=bounds, count=c.move_count)
    count = c.free_count
    used = nb - int(count)
    assert int(host(table)[0].max()) >= 0 and all(
        int(host(table)[0][b, :R.ceil_div(t.shape[0], bs)].max(initial=-1)) < used
        for b, t in enumerate(text))
    step([1, 30, 1, 2, 3, 1, 1, 1, 1, 6])
    # Everything back: every block is on the stack once, no share is left.
    r = binding.paged_free(lens, torch.zeros_like(lens), bs, table, free, count, shares)
    assert int(r.free_count) == nb and sorted(host(free)[0].tolist()) == list(range(nb))
    assert int(shares.abs().sum()) == 0 and int(r.seq_lens.abs().sum()) == 0


@pytest.mark.parametrize("nb,bs,H,D,n,bounds", [
    (5200, 16, 8, 128, 300, True),       # pools past the caches
    (140000, 1, 1, 64, 70000, False),    # more items than a grid has workgroups
])
def test_copy_of_large_pools(nb, bs, H, D, n, bounds):
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(nb, bs, H, D, device=DEV, generator=g).bfloat16() for _ in range(2))
    kb = torch.randn(nb, H, 2, D, device=DEV, generator=g).bfloat16() if bounds else None
    perm = torch.randperm(nb, device=DEV, generator=g)[:2 * n].to(torch.int32)
    src, dst = perm[:n].contiguous(), perm[n:].contiguous()
    want = []
    for x in (k, v, kb):
        want.append(None if x is None else x.clone())
        if x is not None:
            want[-1][dst.long()] = x[src.long()]
    binding.paged_copy(src, dst, k, v, k_bounds=kb)
    for x, w in zip((k, v, kb), want):
        assert x is None or torch.equal(x, w)


def test_upkeep_in_graphs():
    """Captured calls replayed with other contents of their buffers."""
    lens, table, free, count, shares = state(14, 20, 16, 40, 400, 60, empty=8, share=5)
    par, chi = i32([0, 1, 2, 3]), i32([12, 13, 14, 15])
    bufs = dict(t=i32(table), f=i32(free), c=i32([count]), s=i32(shares), l=i32(lens))
    keep = i32(np.zeros(20))
    ws = torch.empty(binding.load_library().mova_paged_compact_workspace_bytes(len(shares)),
                     dtype=torch.uint8, device=DEV)

    def round_(b):
        f = binding.paged_fork(par, chi, 16, b["t"], b["l"], b["f"], b["c"], b["s"])
        r = binding.paged_free(f.seq_lens, keep, 16, b["t"], b["f"], f.free_count, b["s"])
        c = binding.paged_compact(r.seq_lens, 16, b["t"], b["f"], r.free_count, b["s"], workspace=ws)
        return [*f, *r, *c]

    def reset(b, turn):
        keep.copy_(i32(np.maximum(lens - turn * 20, 0)))
        for x, v in zip("tfcsl", (table, free, [count], shares, lens)):
            b[x].copy_(i32(v))
    round_(bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = round_(bufs)
    for turn in range(4):
        reset(bufs, turn)
        graph.replay()
        got = host(*outs)
        reset(bufs, turn)
        want = host(*round_(bufs))
        for g, w in zip(got, want):
            assert np.array_equal(g, w), f"turn {turn}"
