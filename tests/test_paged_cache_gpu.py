"""The paged cache's operators (plan, key / value store, block selection,
decode attention) against plain 64-bit references, and a run of them together
around the value projection."""
import math
import sys

import numpy as np
import pytest
import torch

from mixture_value_projection_amd import binding, inputs
import pagedlib as R
import paritylib as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
FP8 = R.FP8


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(autouse=True)
def _gpu_only():
    assert torch.cuda.is_available(), "GPU test run without a GPU"
    binding.load_library()


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device=DEV)


# ---- plan -------------------------------------------------------------------

def run_plan(cached, new, T, bs, table, free, count):
    dt, df = i32(table), i32(free)
    p = binding.paged_plan(i32(cached), i32(new), T, bs, dt, df, i32([count]))
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (dt, df, *p)]


def check_plan(cached, new, T, bs, table, free, count, what):
    want = R.plan(cached, new, T, bs, table, free, count)
    got = run_plan(cached, new, T, bs, table, free, count)
    for g, w, name in zip(got, [*want[:6], np.array([want[6]])],
                          ("table", "free", "seq_lens", "cu_new", "slots", "positions", "count")):
        assert np.array_equal(g, w), f"{what}: {name}"


def plan_case(seed, B, bs, mb, longest, most_new, ended=0, short=0, extra_rows=0):
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, longest + 1, B)
    new = rng.integers(0, most_new + 1, B)
    new[rng.permutation(B)[:ended]] = -rng.integers(1, 5)
    need = sum(max(0, R.ceil_div(c + n, bs) - R.ceil_div(c, bs)) for c, n in zip(cached, new) if n > 0)
    held = sum(R.ceil_div(c, bs) for c in cached)
    back = sum(R.ceil_div(c, bs) for c, n in zip(cached, new) if n < 0)
    spare = max(0, need - back + 2 - short)
    perm = rng.permutation(held + spare)
    table = np.full((B, mb), -1)
    at = 0
    for b in range(B):
        n = R.ceil_div(cached[b], bs)
        table[b, :n] = perm[at:at + n]
        at += n
    free = np.full(held + spare, -1)
    free[:spare] = perm[at:]
    T = int(np.maximum(new, 0).sum()) + extra_rows
    return cached, new, T, bs, table, free, spare


@pytest.mark.parametrize("seed,kw", [
    (0, dict(B=1, bs=16, mb=4, longest=0, most_new=1)),
    (1, dict(B=1, bs=16, mb=40, longest=300, most_new=300)),
    (2, dict(B=64, bs=16, mb=64, longest=900, most_new=1)),
    (3, dict(B=64, bs=16, mb=64, longest=900, most_new=1, ended=5, extra_rows=9)),
    (4, dict(B=37, bs=24, mb=50, longest=700, most_new=400, ended=4)),
    (5, dict(B=37, bs=24, mb=50, longest=700, most_new=400, ended=4, short=30)),
    (6, dict(B=50, bs=1, mb=300, longest=150, most_new=100, short=200)),
    (7, dict(B=300, bs=8, mb=200, longest=1000, most_new=60, ended=31, short=100, extra_rows=1)),
    (8, dict(B=2048, bs=16, mb=8, longest=100, most_new=20, ended=100, short=50)),
    (9, dict(B=5, bs=128, mb=100, longest=12000, most_new=9000, short=3)),  # past table rows
    (10, dict(B=20, bs=16, mb=64, longest=900, most_new=0, ended=20)),      # everyone ends
])
def test_plan(seed, kw):
    check_plan(*plan_case(seed, **kw), what=str(kw))


def test_plan_few_rows_and_bad_numbers():
    """Tokens past row T, lengths and counts outside their ranges."""
    cached, new, T, bs, table, free, count = plan_case(11, B=30, bs=16, mb=64, longest=500, most_new=50)
    check_plan(cached, new, T // 2, bs, table, free, count, "half the rows")
    check_plan(cached, new, 0, bs, table, free, count, "no rows")
    check_plan(cached, new, T, bs, table, free, 0, "nothing free")
    check_plan(cached, new, T, bs, table, free, -7, "negative count")
    check_plan(cached, new, T, bs, table, free, 10 ** 6, "count above capacity")
    odd = cached.copy()
    odd[3], odd[7] = -50, 10 ** 6
    check_plan(odd, new, T, bs, table, free, count, "lengths out of range")
    big = new.copy()
    big[2:] = 2 ** 31 - 1
    got = run_plan(cached, big, T, bs, table, free, count)
    want = R.plan(cached[:2], big[:2], T, bs, table[:2], free, count)
    assert np.array_equal(got[2][:2], want[2]) and np.array_equal(got[2][2:], cached[2:])
    assert got[3][-1] == 2 ** 31 - 1 and np.array_equal(got[4][:want[3][-1]], want[4][:want[3][-1]])
    assert (got[4][want[3][-1]:] == -1).all()
    # Blocks given back beyond the stack's capacity are dropped.
    check_plan(cached, np.where(np.arange(30) % 2 == 0, -1, new), T, bs, table, free[:20], 18, "drop")
    p = binding.paged_plan(i32([]), i32([]), 3, 16, i32(np.zeros((0, 4))), i32([5, 6]), i32([2]))
    assert p.slot_mapping.tolist() == [-1] * 3 and p.cu_new.tolist() == [0]
    assert p.free_count.tolist() == [2]


# ---- store --------------------------------------------------------------------

def make_pool(rng, nb, bs, H, D, dtype):
    x = torch.from_numpy(rng.standard_normal((nb, bs, H, D), dtype=np.float32))
    if dtype == FP8:
        return (x * 60).clamp(-448, 448).to(FP8)
    return x.to(torch.bfloat16)


def run_slots(rng, nb, bs, runs, T):
    """Slots of `runs` appended runs over distinct blocks, padded with -1 and
    out-of-pool rows to T."""
    pages = iter(rng.permutation(nb))
    slots = []
    for n in runs:
        page, off = int(next(pages)), int(rng.integers(0, bs))
        while n > 0:
            m = min(n, bs - off)
            slots += [page * bs + off + i for i in range(m)]
            n -= m
            off = 0
            if n:
                page = int(next(pages))
    assert len(slots) <= T
    tail = [-1, nb * bs, nb * bs + 77, -(2 ** 40), 2 ** 40]
    return np.array(slots + [tail[i % 5] for i in range(T - len(slots))], dtype=np.int64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("H,D,nb,bs,runs,T", [
    (8, 128, 80, 16, [1] * 64, 64),
    (8, 128, 90, 16, [1, 200, 16, 33, 500], 760),
    (1, 64, 40, 1, [1, 5, 9], 20),
    (3, 64, 70, 24, [60, 1, 1, 700], 770),
    (2, 256, 30, 128, [130, 1, 300], 431),
    (5, 16, 12, 7, [3, 20], 40),
    (2, 80, 12, 8, [1], 1),
])
def test_store(dtype, H, D, nb, bs, runs, T):
    rng = np.random.default_rng(T + D)
    slots = run_slots(rng, nb, bs, runs, T)
    pools = [make_pool(rng, nb, bs, H, D, dtype) for _ in range(2)]
    x = [torch.from_numpy(rng.standard_normal((T, H, D), dtype=np.float32) * 3).to(torch.bfloat16)
         for _ in range(2)]
    scale = [None, None]
    if dtype == FP8:  # one key head far past the range
        scale = [torch.from_numpy(rng.uniform(0.01, 0.03, H).astype(np.float32)) for _ in range(2)]
        scale[0][0] = 1e-3
    before = torch.full((nb, H, 2, D), 7.0, dtype=torch.bfloat16)
    dev = [t.to(DEV) for t in pools]
    kb = before.to(DEV)
    s = torch.as_tensor(slots, device=DEV)
    dsc = [None if t is None else t.to(DEV) for t in scale]
    binding.kv_store_paged(x[0].to(DEV), x[1].to(DEV), dev[0], dev[1], s, k_scale=dsc[0],
                           v_scale=dsc[1], k_bounds=kb)
    torch.cuda.synchronize()
    for i in range(2):
        want = R.store(x[i], pools[i], slots, scale[i])
        assert torch.equal(dev[i].cpu().view(torch.uint8), want.view(torch.uint8)), "kv"[i]
    assert torch.equal(kb.cpu(), R.bounds(R.store(x[0], pools[0], slots, scale[0]), slots, before))
    # Keys or values alone.
    only = pools[1].to(DEV)
    binding.kv_store_paged(None, x[1].to(DEV), None, only, s, v_scale=dsc[1])
    assert torch.equal(only.view(torch.uint8), dev[1].view(torch.uint8))
    only = pools[0].to(DEV)
    binding.kv_store_paged(x[0].to(DEV), None, only, None, s, k_scale=dsc[0])
    assert torch.equal(only.view(torch.uint8), dev[0].view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8], ids=["bf16", "fp8"])
def test_store_special_values(dtype):
    """Every finite e4m3 value and its midpoints, infinities, NaN, signed zeros."""
    e4m3 = torch.arange(0, 127, dtype=torch.uint8).view(FP8).float()
    mid = (e4m3[1:] + e4m3[:-1]) / 2
    vals = torch.cat([e4m3, mid, torch.tensor([448., 460., 464., 480., 1e30, math.inf, math.nan])])
    vals = torch.cat([vals, -vals])
    H, D = 1, 16
    T = R.ceil_div(vals.numel(), D)
    x = torch.zeros(T * D)
    x[:vals.numel()] = vals
    x = x.view(T, H, D).to(torch.bfloat16)
    pool = torch.zeros(T, 1, H, D).to(dtype)
    want = R.store(x, pool, range(T), None)
    dev, kb = pool.to(DEV), torch.zeros(T, H, 2, D, dtype=torch.bfloat16, device=DEV)
    binding.kv_store_paged(x.to(DEV), None, dev, None, torch.arange(T, device=DEV), k_bounds=kb)
    got = dev.cpu().float()
    nan = want.float().isnan()
    assert torch.equal(got.isnan(), nan)
    assert torch.equal(got[~nan], want.float()[~nan])
    assert torch.equal(kb[:, :, 0].cpu().float().nan_to_num(nan=9.0),
                       want.float()[:, 0].to(torch.bfloat16).float().nan_to_num(nan=9.0))


# ---- selection ------------------------------------------------------------------

def make_table(rng, lens, bs, nb, mb):
    perm = rng.permutation(nb)
    table = np.full((len(lens), mb), 2 ** 31 - 1, dtype=np.int64)  # behind the last: not read
    at = 0
    for b, n in enumerate(lens):
        c = min(R.ceil_div(max(n, 0), bs), mb)
        table[b, :c] = perm[at:at + c]
        at += c
    return table


def check_select(q, kb, bs, table, lens, keep, first, last, what):
    want = R.select(q, kb, bs, table, lens, keep, first, last)
    got = binding.block_select(q.to(DEV), kb.to(DEV), bs, i32(table), i32(lens), keep, first, last)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), want), what


SELECT = [
    # lens, Hq, H, D, bs, keep, first, last
    ([1], 4, 1, 128, 16, 1, 0, 1),
    ([700, 0, 33, 5], 32, 8, 128, 16, 8, 1, 2),
    ([5000, 4097], 8, 2, 64, 16, 32, 1, 1),
    ([900, 300], 10, 2, 256, 24, 5, 0, 0),
    ([20000], 16, 1, 128, 8, 100, 2, 4),
    ([3000, 17, 2900], 3, 3, 64, 1, 64, 3, 5),
    ([640] * 9, 8, 8, 128, 32, 20, 1, 1),       # keep == blocks
    ([640] * 9, 20, 4, 128, 32, 33, 1, 1),      # keep > blocks
    ([40000, 100], 4, 1, 64, 2, 1500, 2, 2),    # more blocks and candidates than are held at once
    ([17000], 2, 1, 128, 1, 90, 20, 70),        # only the forced ones
    ([30000, 200, 3000], 8, 2, 128, 4, 16, 1, 3),  # many tiles of blocks, few wanted
    ([60000, 59999], 4, 1, 64, 1, 20, 0, 0),
    ([33000], 4, 2, 256, 1, 40, 17, 20),
    ([-5, 10 ** 6, 48], 6, 2, 64, 16, 6, 1, 1),  # lengths out of range
]


@pytest.mark.parametrize("lens,Hq,H,D,bs,keep,first,last", SELECT)
def test_select(lens, Hq, H, D, bs, keep, first, last):
    rng = np.random.default_rng(len(lens) + D + keep)
    mb = max(1, min(max(R.ceil_div(n, bs) for n in lens), 60000)) + 3
    nb = sum(min(R.ceil_div(max(n, 0), bs), mb) for n in lens) + 2
    table = make_table(rng, lens, bs, nb, mb)
    q = torch.from_numpy(rng.standard_normal((len(lens), Hq, D), dtype=np.float32)).to(torch.bfloat16)
    kb = torch.from_numpy(rng.standard_normal((nb, H, 2, D), dtype=np.float32)).to(torch.bfloat16)
    kb = torch.sort(kb.float(), dim=2).values.to(torch.bfloat16)
    check_select(q, kb, bs, table, lens, keep, first, last, "random")
    # Few distinct scores: whole numbers, so sums are exact and ties many.
    qi = torch.from_numpy(rng.integers(-1, 2, q.shape)).to(torch.bfloat16)
    ki = torch.from_numpy(rng.integers(-1, 2, kb.shape)).to(torch.bfloat16)
    check_select(qi, ki, bs, table, lens, keep, first, last, "ties")
    check_select(torch.zeros_like(q), ki, bs, table, lens, keep, first, last, "all equal")
    # Missing blocks are never chosen, forced or not.
    holes = table.copy()
    holes[:, ::3] = -1
    holes[:, 1::7] = nb
    check_select(q, kb, bs, holes, lens, keep, first, last, "holes")


def test_select_extreme_values():
    rng = np.random.default_rng(5)
    lens, bs, H, D, nb = [600, 590], 8, 2, 64, 160
    table = make_table(rng, lens, bs, nb, 80)
    q = torch.from_numpy(rng.standard_normal((2, 6, D), dtype=np.float32)).to(torch.bfloat16)
    kb = torch.from_numpy(rng.standard_normal((nb, H, 2, D), dtype=np.float32)).to(torch.bfloat16)
    kb[::5, :, :, 3] = math.nan
    kb[1::5, :, 1, 4] = math.inf
    kb[2::5, :, 0, 5] = -math.inf
    kb[3::5] *= 3e38
    check_select(q, kb, bs, table, lens, 40, 1, 1, "extremes")
    q[:, :, 4] = 0  # 0 * inf
    check_select(q, kb, bs, table, lens, 40, 1, 1, "zero times infinity")


def test_select_near_ties():
    """Scores of hundreds that differ in their 30th to 45th bit: the choice is
    that of the 64-bit sums."""
    rng = np.random.default_rng(9)
    for lens, H, D, keep in [([20000, 700], 2, 128, 50), ([9000], 1, 64, 300), ([5000], 4, 256, 7)]:
        bs = 8
        mb = max(R.ceil_div(n, bs) for n in lens)
        nb = sum(R.ceil_div(n, bs) for n in lens) + 1
        table = make_table(rng, lens, bs, nb, mb)
        q = torch.from_numpy(rng.standard_normal((len(lens), 2 * H, D), dtype=np.float32)).to(torch.bfloat16)
        q[:, :, 7] = 2.0 ** -20
        row = np.sort(rng.standard_normal((1, H, 2, D), dtype=np.float32) * 4, axis=2)
        kb = torch.from_numpy(np.repeat(row, nb, axis=0)).to(torch.bfloat16)
        kb[:, :, :, 7] = torch.from_numpy(rng.integers(1, 200, (nb, 1, 1)) * 2.0 ** -8).to(torch.bfloat16)
        check_select(q, kb, bs, table, lens, keep, 1, 1, f"near ties {lens}")


# ---- attention ------------------------------------------------------------------

def make_attention(seed, lens, Hq, H, D, bs, dtype, mb=None, spread=1.0):
    rng = np.random.default_rng(seed)
    mb = mb or max(1, max(R.ceil_div(max(n, 0), bs) for n in lens))
    nb = sum(min(R.ceil_div(max(n, 0), bs), mb) for n in lens) + 2
    a = dict(table=make_table(rng, lens, bs, nb, mb), lens=np.array(lens))
    a["q"] = torch.from_numpy(rng.standard_normal((len(lens), Hq, D), dtype=np.float32)
                              * spread).to(torch.bfloat16)
    a["k"], a["v"] = (make_pool(rng, nb, bs, H, D, dtype) for _ in range(2))
    a["k_scale"] = a["v_scale"] = None
    if dtype == FP8:
        a["k_scale"], a["v_scale"] = (torch.from_numpy(
            rng.uniform(0.01, 0.03, H).astype(np.float32)) for _ in range(2))
    return a


def run_attention(a, window=0, sel=None, scale=None):
    D = a["q"].shape[2]
    dev = {k: (v.to(DEV) if torch.is_tensor(v) else v) for k, v in a.items()}
    lse = torch.full(a["q"].shape[:2], math.nan, device=DEV)
    out = binding.attention_paged(dev["q"], dev["k"], dev["v"], i32(a["table"]), i32(a["lens"]),
                                  D ** -0.5 if scale is None else scale, k_scale=dev["k_scale"],
                                  v_scale=dev["v_scale"], window=window,
                                  sel_blocks=None if sel is None else i32(sel), lse=lse)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def check_attention(a, what, window=0, sel=None, scale=None):
    D = a["q"].shape[2]
    sc = D ** -0.5 if scale is None else scale
    out, lse = run_attention(a, window, sel, scale)
    want, wlse, tol, tlse = R.attention(a["q"], a["k"], a["v"], a["table"], a["lens"], sc,
                                        a["k_scale"], a["v_scale"], window, sel)
    err = (out.double() - want).abs()
    assert (err <= tol).all(), f"{what}: off by {float((err - tol).max()):.3g} too much"
    empty = wlse == -math.inf
    assert torch.equal(lse == -math.inf, empty), what
    assert ((lse.double() - wlse).abs()[~empty] <= tlse[~empty]).all(), f"{what}: lse"
    return out, lse


ATTENTION = [
    # lens, Hq, H, D, bs
    ([1], 1, 1, 64, 16),
    ([1, 0, 2, 15, 16, 17], 32, 8, 128, 16),
    ([31, 32, 33, 63, 64, 65, 127, 129], 8, 2, 128, 16),
    ([2000, 3, 700, 0], 32, 8, 128, 16),
    ([500, 1300], 15, 3, 64, 24),
    ([301, 44], 12, 6, 64, 7),
    ([90, 257], 4, 4, 128, 1),
    ([1500, 80], 16, 1, 128, 64),       # one key head, a full tile of queries
    ([400, 1025], 40, 2, 128, 32),      # groups of 20: more than a tile
    ([700, 10, 333], 8, 2, 256, 16),
    ([1000], 64, 2, 256, 128),
    ([6000], 8, 8, 128, 128),
    ([40] * 70, 8, 4, 64, 8),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("lens,Hq,H,D,bs", ATTENTION)
def test_attention(lens, Hq, H, D, bs, dtype):
    a = make_attention(len(lens) + D, lens, Hq, H, D, bs, dtype)
    say(f"attention {lens[:6]} Hq={Hq} H={H} D={D} bs={bs} {dtype}")
    check_attention(a, "all keys")
    check_attention(a, "window", window=37)
    rng = np.random.default_rng(3)
    mb = a["table"].shape[1]
    sel = rng.integers(-1, mb + 2, (len(lens), H, 9))  # any order, repeats, strangers
    check_attention(a, "listed blocks", sel=sel)
    check_attention(a, "listed blocks in a window", sel=sel, window=max(max(lens) // 3, 1))


def test_large_batches():
    """More requests than a wave has lanes, many of them empty: the shares of
    the workgroups begin anywhere in them."""
    rng = np.random.default_rng(8)
    for B, H, G, D, bs in [(2048, 1, 2, 64, 4), (1500, 4, 1, 64, 8), (65, 2, 3, 128, 16)]:
        lens = rng.integers(0, 40, B) * (rng.random(B) < 0.7)
        lens[-1] = 700
        a = make_attention(B, list(lens), H * G, H, D, bs, torch.bfloat16)
        say(f"batch of {B}")
        check_attention(a, f"batch of {B}")
        kb = torch.zeros(a["k"].shape[0], H, 2, D, dtype=torch.bfloat16)
        kb[:, :, 0], kb[:, :, 1] = a["k"].float().amin(1), a["k"].float().amax(1)
        check_select(a["q"], kb, bs, a["table"], lens, 3, 1, 1, f"batch of {B}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("B,Hq,H,D,bs,longest", [
    (1, 8, 8, 128, 16, 64), (3, 12, 3, 64, 16, 500), (70, 8, 4, 128, 16, 120), (70, 8, 4, 128, 16, 160),
    (300, 4, 2, 64, 8, 900), (5, 40, 2, 256, 16, 90), (1, 32, 8, 128, 16, 320),
    (1, 32, 8, 128, 16, 400), (64, 16, 4, 256, 16, 300), (64, 16, 4, 256, 16, 500),
    (130, 32, 8, 128, 32, 200), (130, 32, 8, 128, 32, 640), (33, 64, 1, 64, 16, 700),
    (17, 96, 2, 128, 16, 500), (260, 8, 4, 64, 8, 1000)])
def test_rows_split_or_whole(B, Hq, H, D, bs, longest, dtype):
    """Batches on either side of where rows stop being split: by the table's
    width, by a window and by the list's length; the same keys in a wider
    table give the same result to rounding."""
    rng = np.random.default_rng(B + longest)
    lens = rng.integers(0, longest + 1, B)
    lens[0] = longest
    a = make_attention(B, list(lens), Hq, H, D, bs, dtype)
    check_attention(a, "narrow table")
    wide = dict(a, table=np.concatenate([a["table"], np.full((B, 4000), -1)], axis=1))
    check_attention(wide, "wide table")
    check_attention(wide, "window", window=min(40, longest))
    sel = rng.integers(-1, R.ceil_div(longest, bs) + 1, (B, H, 2))
    check_attention(wide, "short lists", sel=sel)


def test_one_request_over_all_workgroups():
    """A single row of work (one key head) split into as many parts as there
    are workgroups, and one with a group of query heads above a tile."""
    for Hq, H, D, bs in [(4, 1, 64, 16), (33, 1, 64, 16), (2, 2, 128, 64)]:
        a = make_attention(3, [40000], Hq, H, D, bs, torch.bfloat16)
        check_attention(a, f"Hq={Hq} H={H}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("lens,Hq,H,D,bs", [
    ([3000, 1, 0, 700], 64, 1, 128, 16), ([900, 333], 32, 1, 64, 16), ([5000], 17, 1, 256, 32),
    ([40, 1200], 96, 2, 64, 8), ([2500, 60], 40, 1, 128, 64), ([800, 9], 99, 3, 128, 16),
    ([700] * 9, 96, 3, 256, 16), ([30] * 5, 128, 4, 128, 16), ([100, 2000], 256, 2, 64, 24)])
def test_wide_groups(lens, Hq, H, D, bs, dtype):
    """Groups of more than 16 query heads: several tracks read a key head, side
    by side in a workgroup where their number allows."""
    say(f"wide group {lens[:3]} Hq={Hq} H={H} D={D} {dtype}")
    a = make_attention(Hq + D, lens, Hq, H, D, bs, dtype)
    check_attention(a, "all keys")
    check_attention(a, "window", window=50)
    mb = a["table"].shape[1]
    sel = np.random.default_rng(Hq).integers(-1, mb + 1, (len(lens), H, 12))
    check_attention(a, "listed blocks", sel=sel)


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("lens,Hq,H,D,bs", [
    ([20000], 6, 2, 256, 32), ([9000, 5], 8, 8, 64, 16), ([14000], 5, 1, 128, 16),
    ([12, 30000] + [7] * 62, 32, 8, 128, 16)])
def test_rows_of_many_parts(lens, Hq, H, D, bs, dtype):
    """Long requests by themselves, where several workgroups join a head, and
    one among so many heads that a workgroup joins four."""
    say(f"many parts {lens[:4]} D={D} {dtype}")
    check_attention(make_attention(D + len(lens), lens, Hq, H, D, bs, dtype), "many parts")


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("lens,Hq,H,D,bs,keep", [
    ([100, 1, 0, 37], 8, 4, 128, 16, 90), ([700, 64, 3], 6, 3, 64, 8, 600),
    ([500, 20], 20, 1, 128, 32, 70), ([130, 90, 257], 8, 2, 256, 64, 300),
    ([40] * 80, 4, 4, 64, 16, 20)])
def test_lists_longer_than_the_request(lens, Hq, H, D, bs, keep, dtype):
    """Lists with more entries than the request has blocks: each block once and
    nothing behind, the same from the list's end, a single block as the last
    entry or somewhere between, blocks listed again and again, and nothing."""
    rng = np.random.default_rng(keep)
    B = len(lens)
    a = make_attention(keep, lens, Hq, H, D, bs, dtype)
    blocks = [R.ceil_div(n, bs) for n in lens]

    def lists(fill):
        sel = np.full((B, H, keep), -1)
        for b, n in enumerate(blocks):
            for h in range(H if n else 0):
                fill(sel[b, h], n)
        return sel

    def at(row, where, what):
        row[where] = what

    cases = {
        "front": lists(lambda row, n: at(row, slice(0, n), rng.permutation(n))),
        "end": lists(lambda row, n: at(row, slice(keep - n, keep), rng.permutation(n))),
        "last": lists(lambda row, n: at(row, keep - 1, rng.integers(n))),
        "between": lists(lambda row, n: at(row, rng.integers(keep), rng.integers(n))),
        "again": lists(lambda row, n: at(row, slice(0, keep), rng.integers(0, n, keep))),
        "nothing": lists(lambda row, n: None),
    }
    for what, sel in cases.items():
        say(f"lists of {keep}, {what}")
        check_attention(a, what, sel=sel)
        check_attention(a, what + " in a window", sel=sel, window=30)


def test_attention_bad_tables_and_lengths():
    lens = [300, 200, 150, 10 ** 6, -4]
    a = make_attention(1, lens, 8, 2, 128, 16, torch.bfloat16, mb=20)
    check_attention(a, "lengths out of range")
    nb = a["k"].shape[0]
    a["table"][0, ::2] = -1
    a["table"][1, :] = nb
    a["table"][2, 3:] = -(2 ** 31)
    a["table"][3, 5] = 2 ** 31 - 1
    out, lse = check_attention(a, "holes")
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8], ids=["bf16", "fp8"])
def test_attention_ignores_what_is_masked(dtype):
    """NaN and infinities in rows behind a length, before a window, in blocks
    not listed and in blocks of no request change nothing."""
    a = make_attention(2, [75, 300, 1], 8, 2, 128, 16, dtype)
    sel = np.array([[[0, 4, -1]] * 2, [[18, 3, 7]] * 2, [[0, -1, -1]] * 2])
    runs = [dict(), dict(window=20), dict(sel=sel), dict(sel=sel, window=150)]
    clean = [run_attention(a, **kw) for kw in runs]
    nb, bs = a["k"].shape[:2]
    for kw, want in zip(runs, clean):
        used = np.zeros((nb, bs), dtype=bool)
        for b, n in enumerate(a["lens"]):
            lo = max(0, n - kw["window"]) if "window" in kw else 0
            blocks = range(R.ceil_div(n, bs)) if "sel" not in kw else [j for j in sel[b, 0] if j >= 0]
            for j in blocks:
                for r in range(bs):
                    if lo <= j * bs + r < n:
                        used[a["table"][b, j], r] = True
        bad = dict(a)
        for name in ("k", "v"):
            t = a[name].clone()
            t.view(torch.uint8 if dtype == FP8 else torch.int16)[torch.from_numpy(~used)] = \
                0x7f if dtype == FP8 else (0x7fc0 if name == "k" else 0x7f80)
            bad[name] = t
        got = run_attention(bad, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), kw


def test_attention_large_logits():
    """Softmax over logits of hundreds: one key takes nearly everything."""
    for dtype in (torch.bfloat16, FP8):
        a = make_attention(4, [900, 35], 8, 2, 128, 16, dtype, spread=8.0)
        check_attention(a, "large", scale=1.0)
        check_attention(a, "negative scale", scale=-0.5)
        check_attention(a, "zero scale", scale=0.0)


def test_attention_far_slots():
    """Byte offsets past 32 bits: a pool of 5 GiB, the request in its last blocks."""
    H, D, bs = 8, 128, 64
    nb = (5 << 30) // (bs * H * D * 2)
    a = make_attention(6, [700], 32, H, D, bs, torch.bfloat16)
    n = R.ceil_div(700, bs)
    pages = [nb - 1 - 2 * i for i in range(n)]
    k, v = (torch.zeros(nb, bs, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    old = a["table"][0, :n].copy()
    k[pages], v[pages] = a["k"][old].to(DEV), a["v"][old].to(DEV)
    want, _ = run_attention(a)
    out = binding.attention_paged(a["q"].to(DEV), k, v, i32([pages]), i32([700]), D ** -0.5)
    assert torch.equal(out.cpu(), want)
    # The store and the bounds reach there too.
    rows = torch.randn(3, H, D, device=DEV).to(torch.bfloat16)
    kb = torch.zeros(nb, H, 2, D, dtype=torch.bfloat16, device=DEV)
    s = (nb - 1) * bs
    binding.kv_store_paged(rows, rows, k, v, torch.tensor([s, s + 1, s + 2], device=DEV), k_bounds=kb)
    assert torch.equal(k[nb - 1, :3], rows) and torch.equal(v[nb - 1, :3], rows)
    assert torch.equal(kb[nb - 1, :, 0], rows.amin(0)) and torch.equal(kb[nb - 1, :, 1], rows.amax(0))


# ---- together --------------------------------------------------------------------

class Cache:
    """A small serving loop around one value layer: device state and the plain
    record of every request's keys and values."""

    def __init__(self, dtype, H, D, bs, nb, B, mb, sparse):
        self.dtype, self.H, self.D, self.bs, self.sparse = dtype, H, D, bs, sparse
        self.k, self.v = (torch.zeros(nb, bs, H, D, device=DEV).to(dtype) for _ in range(2))
        self.kb = torch.zeros(nb, H, 2, D, dtype=torch.bfloat16, device=DEV)
        self.table = torch.full((B, mb), -1, dtype=torch.int32, device=DEV)
        self.free = torch.arange(nb, dtype=torch.int32, device=DEV)
        self.count = [i32([nb]), i32([0])]
        self.lens = [torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(2)]
        self.scale = None if dtype != FP8 else torch.full((H,), 1 / 64, device=DEV)

    def step(self, g, x, k, q, new, T, keep=0):
        """One step's calls; returns (plan, value rows, attention out)."""
        p = binding.paged_plan(self.lens[0], new, T, self.bs, self.table, self.free, self.count[0],
                               seq_lens=self.lens[1], free_count_out=self.count[1])
        v = torch.empty(T, self.H, self.D, dtype=torch.bfloat16, device=DEV)
        if self.dtype == FP8:
            binding.value_forward(x, g["router_w"], g["router_b"], g["expert_w"], 4, 2.5, self.H,
                                  self.D, out=v)
            binding.kv_store_paged(k, v, self.k, self.v, p.slot_mapping, k_scale=self.scale,
                                   v_scale=self.scale, k_bounds=self.kb)
        else:
            binding.value_forward_paged(x, g["router_w"], g["router_b"], g["expert_w"], 4, 2.5,
                                        self.v, p.slot_mapping, out=v)
            binding.kv_store_paged(k, None, self.k, None, p.slot_mapping, k_bounds=self.kb)
        sel = None
        if keep:
            sel = binding.block_select(q, self.kb, self.bs, self.table, self.lens[1], keep)
        out = binding.attention_paged(q, self.k, self.v, self.table, self.lens[1], self.D ** -0.5,
                                      k_scale=self.scale, v_scale=self.scale, sel_blocks=sel)
        return p, v, out

    def swap(self):
        self.lens.reverse()
        self.count.reverse()


@pytest.mark.parametrize("dtype,keep", [(torch.bfloat16, 0), (torch.bfloat16, 4), (FP8, 0), (FP8, 3)])
def test_serving_loop(dtype, keep):
    """Requests come, grow, end and give their blocks to others; every step's
    attention equals the plain one over each request's own history."""
    d, E, H, D, bs, B = 256, 8, 2, 64, 8, 5
    rng = np.random.default_rng(7)
    shape = inputs.LayerShape(T=64, d=d, E=E, k=4, n_kv_heads=H, head_dim=D)
    g = P.to_gpu_inputs(inputs.make_layer(shape, 3, torch.bfloat16, "uniform"))
    c = Cache(dtype, H, D, bs, 24, B, 12, keep > 0)
    hist = [[] for _ in range(B)]
    steps = [[30, 5, 0, 1, 17], [1, 1, 9, 1, 1], [1, -1, 1, 1, 1], [1, 40, 1, 1, 1], [-1, 1, 1, 1, 0],
             [33, 1, 1, -1, 1], [1, 1, 1, 2, 1]]
    for i, new in enumerate(steps):
        T = sum(max(n, 0) for n in new) + 2
        x = torch.from_numpy(rng.standard_normal((T, d), dtype=np.float32)).to(DEV, torch.bfloat16)
        k = torch.from_numpy(rng.standard_normal((T, H, D), dtype=np.float32)).to(DEV, torch.bfloat16)
        q = torch.from_numpy(rng.standard_normal((B, 8, D), dtype=np.float32)).to(DEV, torch.bfloat16)
        p, v, out = c.step(g, x, k, q, i32(new), T, keep)
        torch.cuda.synchronize()
        cu, seq = p.cu_new.tolist(), p.seq_lens.tolist()
        for b, n in enumerate(new):
            if n < 0:
                hist[b] = []
            elif seq[b] == len(hist[b]) + n:
                sc = None if c.scale is None else c.scale.cpu()
                kk = R.stored(k[cu[b]:cu[b + 1]].cpu(), dtype, sc)
                vv = R.stored(v[cu[b]:cu[b + 1]].cpu(), dtype, sc)
                hist[b] += [(kk[j], vv[j]) for j in range(n)]
            assert seq[b] == len(hist[b])
        held = sum(R.ceil_div(len(h), bs) for h in hist)
        assert int(p.free_count) == 24 - held, "blocks lost or found"
        nbl = [R.ceil_div(len(h), bs) for h in hist]
        live = [c.table[b, :nbl[b]].tolist() for b in range(B)]
        flat = sum(live, [])
        assert len(set(flat)) == len(flat), "a block in two requests"
        # The histories as a pool of their own.
        mb = max(max(nbl), 1)
        pool = [torch.zeros(B * mb, bs, H, D).to(dtype) for _ in range(2)]
        kb = torch.zeros(B * mb, H, 2, D, dtype=torch.bfloat16)
        tab = np.arange(B * mb).reshape(B, mb)
        for b, h in enumerate(hist):
            for j, row in enumerate(h):
                for s in range(2):
                    pool[s].view(torch.uint8)[b * mb + j // bs, j % bs] = row[s].view(torch.uint8)
            for j in range(nbl[b]):
                rows = pool[0][b * mb + j, :min(bs, len(h) - j * bs)].float()
                kb[b * mb + j, :, 0], kb[b * mb + j, :, 1] = rows.amin(0), rows.amax(0)
        sel = R.select(q.cpu(), kb, bs, tab, seq, keep, 1, 1) if keep else None
        sc = None if c.scale is None else c.scale.cpu()
        want, _, tol, _ = R.attention(q.cpu(), pool[0], pool[1], tab, seq, D ** -0.5, sc, sc, 0, sel)
        assert ((out.cpu().double() - want).abs() <= tol).all(), f"step {i}"
        c.swap()
    assert any(len(h) for h in hist)


@pytest.mark.parametrize("dtype,keep", [(torch.bfloat16, 0), (torch.bfloat16, 4), (FP8, 3)])
def test_captured_decode_steps(dtype, keep):
    """Two decode steps (the double-buffered lengths) captured in one graph and
    replayed while the lengths grow, against the same steps run eagerly."""
    d, E, H, D, bs, B, mb, nb = 256, 8, 2, 64, 8, 6, 16, 80
    shape = inputs.LayerShape(T=64, d=d, E=E, k=4, n_kv_heads=H, head_dim=D)
    g = P.to_gpu_inputs(inputs.make_layer(shape, 3, torch.bfloat16, "uniform"))
    gen = torch.Generator(device=DEV).manual_seed(5)
    prompt = [3, 40, 17, 1, 0, 8]

    def rows(n, w):
        return torch.randn(n, *w, device=DEV, generator=gen).to(torch.bfloat16)

    first = (rows(sum(prompt), (d,)), rows(sum(prompt), (H, D)), rows(B, (8, D)))
    xs = [(rows(B, (d,)), rows(B, (H, D)), rows(B, (8, D))) for _ in range(10)]
    one = i32([1] * B)
    caches, feeds, results = [], [], []
    for _ in range(2):
        c = Cache(dtype, H, D, bs, nb, B, mb, keep > 0)
        c.step(g, *first, i32(prompt), sum(prompt), keep)
        c.swap()
        caches.append(c)
    eager, live = caches
    for x in xs:
        results.append(eager.step(g, *x, one, B, keep)[2].clone())
        eager.swap()
    feed = [tuple(t.clone() for t in xs[0]) for _ in range(2)]
    side = torch.cuda.Stream()
    warm = Cache(dtype, H, D, bs, nb, B, mb, keep > 0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm.step(g, *feed[0], one, B, keep)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = []
        for i in range(2):
            outs.append(live.step(g, *feed[i], one, B, keep)[2])
            live.swap()
    for r in range(5):
        for i in range(2):
            for dst, src in zip(feed[i], xs[2 * r + i]):
                dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], results[2 * r + i]), f"replay {r} step {i}"
        # The program's own work between replays, on the operators' scratch too.
        warm.step(g, *xs[r], one, B, keep)
        torch.cuda.synchronize()
    assert torch.equal(live.lens[0], eager.lens[0]) and torch.equal(live.table, eager.table)


def test_two_streams_at_once():
    """Two attention calls in flight on two streams, each with its workspace."""
    a = [make_attention(s, [3000, 1500], 32, 8, 128, 16, torch.bfloat16) for s in (1, 2)]
    want = [run_attention(x)[0] for x in a]
    dev = [{k: (v.to(DEV) if torch.is_tensor(v) else v) for k, v in x.items()} for x in a]
    tabs = [(i32(x["table"]), i32(x["lens"])) for x in a]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(binding.attention_paged(dev[i]["q"], dev[i]["k"], dev[i]["v"], *tabs[i],
                                                       128 ** -0.5))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o.cpu(), want[i])


def test_two_graphs_share_a_workspace():
    """Two captured sparse steps over one workspace, replayed in turns with
    eager calls on it between them."""
    a = [make_attention(s, lens, 16, 4, 128, 16, torch.bfloat16)
         for s, lens in ((1, [3000, 40, 900]), (2, [77, 2500, 0]))]
    dev = [{k: (v.to(DEV) if torch.is_tensor(v) else v) for k, v in x.items()} for x in a]
    tabs = [(i32(x["table"]), i32(x["lens"])) for x in a]
    kb = []
    for x in dev:
        t = torch.empty(x["k"].shape[0], 4, 2, 128, dtype=torch.bfloat16, device=DEV)
        t[:, :, 0], t[:, :, 1] = x["k"].float().amin(1), x["k"].float().amax(1)
        kb.append(t)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)

    def step(i, ws):
        sel = binding.block_select(dev[i]["q"], kb[i], 16, *tabs[i], 6, workspace=ws)
        return sel, binding.attention_paged(dev[i]["q"], dev[i]["k"], dev[i]["v"], *tabs[i],
                                            128 ** -0.5, sel_blocks=sel, workspace=ws)

    want = [[t.clone() for t in step(i, None)] for i in range(2)]
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(i, ws))
        graphs.append(g)
    for r in range(4):
        for i in (0, 1, 1, 0):
            for t in outs[i]:
                t.zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(outs[i], want[i])), (r, i)
            step(1 - i, ws)
            torch.cuda.synchronize()
