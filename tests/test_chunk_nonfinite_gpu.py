"""Chunk attention over values that are infinite or NaN, or whose sums pass the
largest number, in many rows at once, against the plain 64-bit reference: such
values show in the rows that see them and in no others, and cost a call a small
factor, not a round trip to memory a key and row."""
import math

import numpy as np
import pytest
import torch

from mixture_value_projection_amd import binding
import blockslib as R
from test_chunk_attention_gpu import BF16, DEV, FP8, Case, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_only():
    assert torch.cuda.is_available(), "GPU test run without a GPU"
    binding.load_library()


def spoil(c, seed, n, kinds):
    """n elements of the values at random positions of random requests become
    infinite or NaN; returns [(request, position, head, channel, value)]."""
    rng = np.random.default_rng(seed)
    H, D = c.v.shape[2:]
    out = []
    for _ in range(n):
        b = int(rng.choice([x for x in range(len(c.lens)) if c.lens[x] > 0]))
        p, h, d = int(rng.integers(c.lens[b])), int(rng.integers(H)), int(rng.integers(D))
        page = c.table[b, p // c.bs]
        if not 0 <= page < c.v.shape[0]:
            continue
        x = float(rng.choice(kinds))
        if c.v.dtype == FP8:
            c.v.view(torch.uint8)[page, p % c.bs, h, d] = 0x7f
            x = math.nan  # (e4m3 has no infinity)
        else:
            c.v[page, p % c.bs, h, d] = x
        out.append((b, p, h, d, x))
    return out


def check(c, bad, what):
    """Against the reference of the values with zeros in place of the bad ones,
    and in the channels of rows that see such: plus and minus infinity, NaN."""
    clean = c.v.clone()
    if clean.dtype == FP8:
        raw = clean.view(torch.uint8)
        raw[(raw & 0x7f) == 0x7f] = 0
    else:
        clean[~torch.isfinite(clean.float())] = 0
    before = torch.full_like(c.q, -3.0)
    want, want_lse, tol, tol_lse = R.chunk(c.q, c.k, clean, c.table, c.cached, c.lens, c.cu, c.scale,
                                           c.ks, c.vs, c.window, before)
    T, Hq, _ = c.q.shape
    G = Hq // c.v.shape[2]
    up, down = torch.zeros(want.shape, dtype=torch.bool), torch.zeros(want.shape, dtype=torch.bool)
    for b, p, h, d, x in bad:
        for t in range(int(c.cu[b]), int(c.cu[b + 1])):
            at = int(c.cached[b]) + t - int(c.cu[b])
            if at < c.lens[b] and p <= at and (not c.window or p > at - c.window):
                up[t, h * G:(h + 1) * G, d] |= not x == -math.inf
                down[t, h * G:(h + 1) * G, d] |= not x == math.inf
    out, lse = before.to(DEV), torch.full((T, Hq), math.nan, device=DEV)
    c.run(out=out, lse=lse)
    got, got_lse = out.cpu().double(), lse.cpu().double()
    assert bool((got[up & down].isnan()).all()), f"{what}: NaN"
    assert bool((got[up & ~down] == math.inf).all()), f"{what}: infinity"
    assert bool((got[down & ~up] == -math.inf).all()), f"{what}: minus infinity"
    rest = ~(up | down)
    within = ((got - want).abs() <= tol) | ~rest
    print(f"{what}: {int((up | down).sum())} infinite or NaN, {int((~within).sum())} others off",
          flush=True)
    assert bool(within.all()), what
    same = (want_lse == got_lse) | (want_lse.isnan() & got_lse.isnan())
    assert bool((same | ((got_lse - want_lse).abs() <= tol_lse)).all()), f"{what}: lse"


SHAPES = [
    # Hq, H, D, bs, dtype
    (8, 2, 128, 16, BF16), (8, 2, 128, 16, FP8), (6, 3, 64, 24, BF16), (15, 3, 64, 8, FP8),
    (4, 2, 256, 64, BF16), (8, 2, 256, 16, FP8), (33, 1, 64, 48, BF16), (4, 4, 128, 1, BF16),
]
ALL = (math.inf, -math.inf, math.nan)


@pytest.mark.parametrize("Hq,H,D,bs,dtype", SHAPES)
@pytest.mark.parametrize("window", [0, 90])
def test_many_rows(Hq, H, D, bs, dtype, window):
    c = Case(1, [700, 0, 33], [200, 150, 40], Hq, H, D, bs, dtype, window=window, padding=2)
    check(c, spoil(c, 5, 12, ALL), f"many rows {Hq}/{H}/{D} window {window}")


@pytest.mark.parametrize("Hq,H,D,bs,dtype", SHAPES)
@pytest.mark.parametrize("window", [0, 90])
def test_few_rows(Hq, H, D, bs, dtype, window):
    c = Case(2, [700, 0, 33, 130, 64, 9], [1, 4, 2, 1, 0, 3], Hq, H, D, bs, dtype, window=window,
             padding=1)
    check(c, spoil(c, 6, 20, ALL), f"few rows {Hq}/{H}/{D} window {window}")


@pytest.mark.parametrize("Hq,H,D,bs,dtype", SHAPES[:6])
def test_rows_split_among_workgroups(Hq, H, D, bs, dtype):
    """A part of the keys to each workgroup, with the bad values in some."""
    for new in (2, 40):
        c = Case(3, [6000], [new], Hq, H, D, bs, dtype, missing=3)
        check(c, spoil(c, new, 3, ALL), f"split {new} {Hq}/{H}/{D}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [[3, 1, 2], [90, 40, 200]])
def test_sums_past_the_largest_number(D, new):
    """Values near the largest in some channels, ordinary ones in others, and
    infinite ones beside them."""
    c = Case(4, [500, 9, 64], new, 4, 2, D, 16, lean=0.0)
    big = torch.finfo(BF16).max
    c.v[..., 3] = big
    c.v[..., 40] = torch.where(c.v[..., 40] > 0, big, -big).to(BF16)
    c.v[..., 41] = torch.where(c.v[..., 41] > 0, big, c.v[..., 41].float()).to(BF16)
    check(c, [], f"large {D} {new}")
    check(c, spoil(c, 7, 4, ALL), f"large and infinite {D} {new}")


@pytest.mark.parametrize("new", [[2, 1], [60, 90]])
def test_other_channels_of_a_weight_of_nothing(new):
    """An infinite value whose weight is far below the smallest number: its own
    channel may be NaN, the others are as without it."""
    c = Case(5, [200, 40], new, 4, 2, 64, 16, lean=0.0, scale=1.0)
    c.q[..., 0] = 8.0
    c.k[..., 0] = 0.0
    for b in range(2):
        c.k[c.table[b, 0], 3, :, 0] = -100.0  # a logit lower by 800
        c.v[c.table[b, 0], 3, :, 7] = math.inf
    clean = Case(5, [200, 40], new, 4, 2, 64, 16, lean=0.0, scale=1.0)
    clean.q, clean.k = c.q, c.k
    want, _, tol, _ = clean.want(None)
    got = c.run().cpu().double()
    rest = [d for d in range(64) if d != 7]
    assert bool(((got - want).abs() <= tol)[..., rest].all())


def test_negative_and_no_scale():
    for scale in (-0.2, 0.0):
        c = Case(6, [100, 0], [70, 3], 8, 2, 128, 16)
        c.scale = scale
        check(c, spoil(c, 8, 6, ALL), f"scale {scale}")


def time_of(f):
    for _ in range(2):
        f()
    times = []
    for _ in range(3):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_a_bad_value_costs_a_small_factor(dtype):
    """A value that all rows of a prompt of 1536 tokens see.  (A round trip to
    memory for each key and row would take a hundred times the call.)"""
    n, H, Hq, D, bs = 1536, 8, 32, 128, 16
    g = torch.Generator(device=DEV).manual_seed(0)
    q = torch.randn(n, Hq, D, generator=g, device=DEV).to(BF16)
    k, v = (torch.randn(n // bs, bs, H, D, generator=g, device=DEV).to(dtype) for _ in range(2))
    bad = v.clone()
    if dtype == FP8:
        bad.view(torch.uint8)[0, 0] = 0x7f
    else:
        bad[0, 0] = math.inf
    table, zero, lens, cu = i32(np.arange(n // bs)[None]), i32([0]), i32([n]), i32([0, n])
    out = torch.empty_like(q)
    ws = torch.empty(binding.attention_chunk_workspace_bytes(n, 1, Hq, H, D, n // bs, bs),
                     dtype=torch.uint8, device=DEV)
    plain, spoiled = (time_of(lambda x=x: binding.attention_chunk_paged(
        q, k, x, table, zero, lens, cu, D ** -0.5, out=out, workspace=ws)) for x in (v, bad))
    print(f"{plain * 1e3:.0f} us, {spoiled * 1e3:.0f} with a bad value", flush=True)
    assert spoiled <= 25 * plain
