"""Chunk attention over the paged cache against a plain 64-bit reference."""
import math
import sys

import numpy as np
import pytest
import torch

from mixture_value_projection_amd import binding
import blockslib as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
FP8 = R.FP8
BF16 = torch.bfloat16


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(autouse=True)
def _gpu_only():
    assert torch.cuda.is_available(), "GPU test run without a GPU"
    binding.load_library()


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device=DEV)


class Case:
    """Inputs on the CPU, for the given cached and new tokens per request."""

    def __init__(self, seed, cached, new, Hq, H, D, bs, dtype=BF16, window=0, refused=(), missing=0,
                 padding=0, ahead=0, width=None, lean=1.0, scale=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.bs, self.window, self.scale = bs, window, scale or D ** -0.5
        self.cached, new = np.array(cached), np.array(new)
        total = self.cached + new
        for b in refused:
            total[b] = self.cached[b]
        self.lens = total
        self.cu = ahead + np.concatenate([[0], np.cumsum(new)])
        T = int(self.cu[-1]) + padding
        need = [R.ceil_div(int(n), bs) for n in total]
        pool = sum(need) + 2
        perm = rng.permutation(pool)
        self.table = np.full((len(need), width or max(1, max(need))), -1)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        for _ in range(missing):
            b = int(rng.integers(len(need)))
            if need[b]:
                self.table[b, int(rng.integers(need[b]))] = rng.choice([-1, pool, pool + 7, -100])
        self.q = torch.randn(T, Hq, D, generator=g).to(BF16)
        k = torch.randn(pool, bs, H, D, generator=g) + lean * torch.randn(pool, 1, H, D, generator=g)
        v = torch.randn(pool, bs, H, D, generator=g)
        self.ks = self.vs = None
        if dtype == FP8:
            self.ks = (1 + torch.rand(H, generator=g)) / 64
            self.vs = (1 + torch.rand(H, generator=g)) / 64
            k, v = k / self.ks[:, None], v / self.vs[:, None]
            k, v = k.clamp(-448, 448), v.clamp(-448, 448)
        self.k, self.v = k.to(dtype), v.to(dtype)

    def want(self, before):
        return R.chunk(self.q, self.k, self.v, self.table, self.cached, self.lens, self.cu,
                       self.scale, self.ks, self.vs, self.window, before)

    def args(self):
        return [self.q.to(DEV), self.k.to(DEV), self.v.to(DEV), i32(self.table), i32(self.cached),
                i32(self.lens), i32(self.cu), self.scale]

    def kw(self):
        return dict(k_scale=None if self.ks is None else self.ks.to(DEV),
                    v_scale=None if self.vs is None else self.vs.to(DEV), window=self.window)

    def run(self, **more):
        return binding.attention_chunk_paged(*self.args(), **self.kw(), **more)

    def check(self, what):
        T, Hq, _ = self.q.shape
        before = torch.full_like(self.q, -3.0)
        out = before.to(DEV)
        lse = torch.full((T, Hq), math.nan, device=DEV)
        self.run(out=out, lse=lse)
        torch.cuda.synchronize()
        want, want_lse, tol, tol_lse = self.want(before)
        got, got_lse = out.cpu().double(), lse.cpu().double()
        off = (got - want).abs()
        worst = float((off / tol.clamp(min=1e-30)).amax()) if off.numel() else 0.0
        say(f"{what}: worst {worst:.3f} of the tolerance")
        assert torch.isfinite(got).all(), what
        assert bool((off <= tol).all()), f"{what}: {worst}"
        same = (want_lse == got_lse) | (want_lse.isnan() & got_lse.isnan())
        near = (got_lse - want_lse).abs() <= tol_lse
        assert bool((same | near).all()), f"{what}: lse"
        return out


def put(pool, where, value):
    """pool[where] = value (8-bit: NaN)."""
    if pool.dtype == FP8:
        pool.view(torch.uint8)[where] = 0x7f
    else:
        pool[where] = value


SHAPES = [
    # Hq, H, D, bs, dtype
    (32, 8, 128, 16, BF16), (32, 8, 128, 32, FP8), (15, 3, 64, 24, BF16), (15, 3, 64, 8, FP8),
    (4, 2, 256, 64, BF16), (8, 2, 256, 16, FP8), (2, 2, 128, 128, BF16), (16, 1, 128, 1, BF16),
    (33, 1, 64, 48, BF16), (130, 1, 64, 16, BF16), (7, 7, 64, 16, FP8), (300, 1, 64, 16, BF16),
]


@pytest.mark.parametrize("Hq,H,D,bs,dtype", SHAPES)
def test_ragged(Hq, H, D, bs, dtype):
    """One token, prompts without a cache, chunks that end inside blocks and
    tiles, requests without new tokens, refused ones, rows behind the last."""
    Case(1, [0, 130, 77, 500, 64, 0, 1], [1, 19, 64, 1, 0, 130, 3], Hq, H, D, bs, dtype,
         refused=[3], padding=5).check(f"ragged {Hq}/{H}/{D} {dtype}")


@pytest.mark.parametrize("Hq,H,D,bs,dtype", SHAPES)
@pytest.mark.parametrize("window", [1, 37, 200])
def test_window(Hq, H, D, bs, dtype, window):
    Case(2, [300, 0, 90], [70, 65, 2], Hq, H, D, bs, dtype, window=window).check(
        f"window {window} {Hq}/{H}/{D}")


@pytest.mark.parametrize("Hq,H,D,bs,dtype", SHAPES)
def test_missing_blocks(Hq, H, D, bs, dtype):
    """Table entries that name no block: their keys take no part."""
    Case(3, [200, 0, 33], [40, 100, 5], Hq, H, D, bs, dtype, missing=6, padding=1, ahead=3).check(
        f"missing {Hq}/{H}/{D}")


@pytest.mark.parametrize("Hq,H,D,bs,dtype", [s for s in SHAPES if s[1] <= 3])
def test_few_rows_long_cache(Hq, H, D, bs, dtype):
    """Rows whose keys are split among workgroups."""
    Case(4, [9001, 3], [3, 1], Hq, H, D, bs, dtype).check(f"long {Hq}/{H}/{D}")


@pytest.mark.parametrize("Hq,H,D,bs,dtype,new,cached", [
    (8, 2, 128, 16, BF16, 700, 0), (8, 2, 128, 16, FP8, 300, 1111), (4, 1, 256, 32, BF16, 333, 500),
    (6, 2, 64, 24, BF16, 900, 77), (1, 1, 128, 16, BF16, 1500, 10), (5, 1, 256, 64, FP8, 257, 1),
])
def test_prompt(Hq, H, D, bs, dtype, new, cached):
    Case(5, [cached], [new], Hq, H, D, bs, dtype).check(f"prompt {new} after {cached}")


@pytest.mark.parametrize("new", [1, 2, 7, 8, 9, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("G", [1, 4])
def test_chunk_sizes(new, G):
    """Around the edges of the row tiles, and keys around those of the key tiles."""
    for cached in (0, 63 - min(new, 63), 64, 127):
        Case(new, [cached], [new], 2 * G, 2, 128, 16).check(f"{new} after {cached}, group {G}")


def test_many_requests():
    rng = np.random.default_rng(0)
    Case(6, rng.integers(0, 90, 300), rng.integers(0, 5, 300), 4, 2, 64, 16, padding=2).check("300")
    Case(7, rng.integers(0, 9, 2048), rng.integers(0, 3, 2048), 2, 1, 64, 8).check("2048")
    new = rng.integers(0, 3, 129)
    new[[5, 70]] = 200
    Case(8, rng.integers(0, 1000, 129), new, 8, 2, 128, 16, FP8).check("mixed")


def test_lengths_outside_the_table():
    """Lengths below 0 and beyond the table row count as its ends, and cu_new
    beyond T as T."""
    c = Case(9, [20, 40, 0], [5, 9, 6], 4, 2, 64, 16)
    c.lens = np.array([-7, 1000, 6])      # nothing; the whole row of 4 blocks
    c.cached = np.array([-3, 40, -5])     # 0 for the third
    c.cu = np.array([0, 5, 14, 900])
    c.check("outside")


def test_decode_rows_agree_with_one_token_attention():
    """A chunk of one token is what attention_paged computes."""
    c = Case(10, [700, 0, 64, 1000], [1, 1, 1, 1], 32, 8, 128, 16)
    args = c.args()
    one = binding.attention_paged(args[0], args[1], args[2], args[3], args[5], c.scale)
    out = c.run()
    _, _, tol, _ = c.want(None)
    assert bool(((one.double() - out.double()).abs().cpu() <= 2 * tol).all())


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_values_that_take_no_part(dtype, D, what):
    """NaN (and infinity) behind the last token, in blocks that no row holds,
    outside the window and in keys ahead of a row's own position: none shows in
    a row that does not see it."""
    bad = what  # (e4m3 has no infinity)
    clean = Case(11, [100, 5], [40, 70], 8, 2, D, 16, dtype, window=60)
    for first in (0, 10, 33):  # rows from here on see the bad key
        c = Case(11, [100, 5], [40, 70], 8, 2, D, 16, dtype, window=60)
        for b in range(2):
            n = int(c.lens[b])
            p = int(c.cached[b]) + first
            for pos in (p, 0):
                page = c.table[b, pos // 16]
                put(c.v, (page, pos % 16), bad)
                put(c.k, (page, pos % 16), bad)
            if n % 16:
                page = c.table[b, n // 16]
                put(c.k, (page, slice(n % 16, None)), bad)
                put(c.v, (page, slice(n % 16, None)), bad)
        used = set(c.table[c.table >= 0].tolist())
        for page in set(range(c.k.shape[0])) - used:
            put(c.k, page, bad)
            put(c.v, page, bad)
        out = c.run().cpu()
        ref = clean.run().cpu()
        want, _, tol, _ = clean.want(None)
        for b in range(2):
            for j in range(int(c.cu[b + 1] - c.cu[b])):
                at = int(c.cached[b]) + j
                sees = {p for p in (int(c.cached[b]) + first, 0) if at - 60 < p <= at}
                t = int(c.cu[b]) + j
                if not sees:
                    off = (out[t].double() - want[t]).abs()
                    assert bool((off <= tol[t]).all()), f"row {t} of request {b}, from {first}"
        assert torch.isfinite(ref).all()


def test_infinite_values_that_take_part():
    """An infinite value makes its channel infinite in the rows that see it."""
    c = Case(12, [50], [30], 4, 1, 64, 16, lean=0.0)
    p = 60
    c.v[c.table[0, p // 16], p % 16, 0, 5] = math.inf
    c.v[c.table[0, p // 16], p % 16, 0, 9] = -math.inf
    out = c.run().cpu().float()
    for j in range(30):
        seen = 50 + j >= p
        assert bool((out[j, :, 5] == math.inf).all()) == seen
        assert bool((out[j, :, 9] == -math.inf).all()) == seen
        rest = [d for d in range(64) if d not in (5, 9)]
        assert torch.isfinite(out[j][:, rest]).all()
        if not seen:
            assert torch.isfinite(out[j]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_near_the_largest(D):
    """Finite values as large as bf16 holds: sums of them stay finite."""
    c = Case(13, [500], [40], 4, 2, D, 16, lean=0.0)
    big = torch.finfo(BF16).max
    c.v = torch.where(c.v > 0, big, -big).to(BF16)
    c.v[:, :, 0] = big
    out = c.run().cpu().double()
    want, _, tol, _ = c.want(None)
    assert bool(((out - want).abs() <= tol).all())


def test_rows_whose_logits_are_all_minus_infinity():
    """Zeros, and an lse of -infinity."""
    c = Case(14, [30], [20], 4, 2, 64, 16, lean=0.0)
    c.q[:] = 0
    c.q[:, :, 0] = 1
    c.k[..., 0] = -math.inf
    lse = torch.zeros(20, 4, device=DEV)
    out = c.run(lse=lse)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_large_logits():
    """Logits of some thousands, differing between neighbouring tiles."""
    c = Case(15, [700, 0], [90, 70], 8, 2, 128, 16, lean=4.0, scale=8.0)
    c.check("large logits")
    c = Case(16, [700, 0], [90, 70], 8, 2, 128, 16, FP8, lean=4.0, scale=-3.0)
    c.check("negative scale")


def test_repeats_bit_for_bit():
    c = Case(17, [3000, 10, 0], [5, 300, 70], 8, 2, 128, 16)
    args, kw = c.args(), c.kw()
    first = binding.attention_chunk_paged(*args, **kw)
    for _ in range(3):
        assert torch.equal(first, binding.attention_chunk_paged(*args, **kw))


def test_given_output_and_workspace():
    c = Case(18, [900, 10], [5, 70], 8, 2, 128, 16)
    T, Hq, D = c.q.shape
    n = binding.attention_chunk_workspace_bytes(T, 2, Hq, 2, D, c.table.shape[1], 16)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    out = torch.empty(T, Hq, D, dtype=BF16, device=DEV)
    got = c.run(out=out, workspace=ws)
    assert got is out and torch.equal(out, c.run())


def test_another_stream():
    c = Case(19, [900, 10], [5, 70], 8, 2, 128, 16)
    want = c.run()
    args, kw = c.args(), c.kw()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = binding.attention_chunk_paged(*args, **kw)
    s.synchronize()
    assert torch.equal(got, want)


def test_graphs_on_one_workspace():
    """Two captured calls that share a workspace, replayed in turn with eager
    work between and with lengths that change under them."""
    a = Case(20, [2000, 10], [5, 70], 8, 2, 128, 16)
    b = Case(21, [0, 700, 3], [200, 4, 1], 8, 2, 64, 16, FP8)
    calls = []
    for c in (a, b):
        args, kw = c.args(), c.kw()
        T, Hq, D = c.q.shape
        calls.append([c, args, kw, torch.empty_like(args[0]),
                      binding.attention_chunk_workspace_bytes(T, len(c.lens), Hq, 2, D,
                                                              c.table.shape[1], 16)])
    ws = torch.empty(max(x[4] for x in calls), dtype=torch.uint8, device=DEV)
    graphs = []
    for c, args, kw, out, _ in calls:
        binding.attention_chunk_paged(*args, **kw, out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.attention_chunk_paged(*args, **kw, out=out, workspace=ws)
        graphs.append(g)
    for turn in range(4):
        for (c, args, kw, out, _), g in zip(calls, graphs):
            if turn == 2:  # fewer tokens cached
                args[4].copy_(args[4] // 2)
                args[5].copy_(args[4] + i32(np.diff(c.cu)))
            out.fill_(7)
            g.replay()
            torch.cuda.synchronize()
            want = binding.attention_chunk_paged(*args, **kw)
            assert torch.equal(out, want), f"turn {turn}"
