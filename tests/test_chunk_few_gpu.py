"""Chunk attention of requests with few rows, whose tiles another kernel reads
than those of many, and of both in one batch, against the plain 64-bit
reference; the inputs and checks are those of test_chunk_attention_gpu."""
import math

import numpy as np
import pytest
import torch

from mixture_value_projection_amd import binding
from test_chunk_attention_gpu import BF16, DEV, FP8, Case, i32, put

pytestmark = pytest.mark.gpu

# Key heads in fours, twos and single ones; a group that fills sixteen rows, one
# that does not divide them, and one larger than them.
SHAPES = [
    # Hq, H, D, bs, dtype
    (32, 8, 128, 16, BF16), (8, 4, 64, 24, FP8), (6, 2, 256, 16, BF16), (15, 3, 128, 8, FP8),
    (20, 1, 64, 32, BF16), (12, 4, 256, 64, FP8), (14, 2, 64, 1, BF16), (64, 1, 128, 16, FP8),
]


@pytest.fixture(autouse=True)
def _gpu_only():
    assert torch.cuda.is_available(), "GPU test run without a GPU"
    binding.load_library()


def batch(G, most):
    """New tokens with most * G rows at most, among requests of few."""
    return [1, max(most // G, 1), 0, 1, min(2, max(most // G, 1)), 1, 1, 1]


@pytest.mark.parametrize("Hq,H,D,bs,dtype", SHAPES)
def test_single_tokens_and_drafts(Hq, H, D, bs, dtype):
    Case(1, [0, 130, 77, 500, 64, 15, 1, 16], batch(Hq // H, 16), Hq, H, D, bs, dtype, refused=[3],
         padding=3).check(f"few {Hq}/{H}/{D} {dtype}")


@pytest.mark.parametrize("Hq,H,D,bs,dtype", SHAPES)
@pytest.mark.parametrize("window", [1, 40])
def test_window_and_missing_blocks(Hq, H, D, bs, dtype, window):
    Case(2, [300, 33, 0, 8, 64, 0, 31, 700], batch(Hq // H, 64), Hq, H, D, bs, dtype, window=window,
         missing=5, ahead=2).check(f"window {window} {Hq}/{H}/{D}")


@pytest.mark.parametrize("G", [1, 3, 4, 16])
@pytest.mark.parametrize("rows", [16, 17, 48, 63, 64, 65, 80, 129])
def test_rows_around_the_bound(rows, G):
    """One request around the number of rows where the other kernel takes over,
    among single tokens: both read the batch."""
    new = [1, -(-rows // G), 1, 0, 1, 1, 1, 1, 1]
    Case(3, [70, 90, 0, 5, 64, 63, 300, 16, 128], new, 2 * G, 2, 128, 16).check(f"{rows} rows of {G}")


@pytest.mark.parametrize("Hq,H,D,dtype", [(4, 1, 64, BF16), (2, 2, 128, FP8), (4, 4, 256, BF16)])
def test_rows_split_among_all_workgroups(Hq, H, D, dtype):
    """More parts to a row than a wave has lanes."""
    Case(4, [40000], [3], Hq, H, D, 16, dtype).check(f"one long {Hq}/{H}/{D}")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows_split_among_all_workgroups(D):
    Case(5, [33000], [70], 1, 1, D, 32).check(f"70 tokens {D}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H", [1, 4])
def test_values_near_the_largest(D, H):
    c = Case(6, [500, 9, 0, 40], [2, 1, 1, 3], 4 * H, H, D, 16, lean=0.0)
    big = torch.finfo(BF16).max
    c.v = torch.where(c.v > 0, big, -big).to(BF16)
    c.v[:, :, 0] = big
    out = c.run().cpu().double()
    want, _, tol, _ = c.want(None)
    assert bool(((out - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_that_take_no_part(dtype, D):
    """NaN in keys ahead of a row's position, before its window, behind the last
    token and in blocks of no row."""
    kw = dict(window=50)
    shape = ([100, 5, 64, 0], [4, 3, 1, 4], 8, 2, D, 16, dtype)
    clean = Case(7, *shape, **kw)
    want, _, tol, _ = clean.want(None)
    for first in range(4):  # rows from here on see the bad key
        c = Case(7, *shape, **kw)
        for b in range(4):
            p, n = int(c.cached[b]) + first, int(c.lens[b])
            for pos in {p, 0}:
                if pos < n:
                    put(c.v, (c.table[b, pos // 16], pos % 16), math.nan)
                    put(c.k, (c.table[b, pos // 16], pos % 16), math.nan)
            if n % 16:
                put(c.k, (c.table[b, n // 16], slice(n % 16, None)), math.nan)
                put(c.v, (c.table[b, n // 16], slice(n % 16, None)), math.nan)
        used = set(c.table[c.table >= 0].tolist())
        for page in set(range(c.k.shape[0])) - used:
            put(c.k, page, math.nan)
            put(c.v, page, math.nan)
        out = c.run().cpu().double()
        seen = 0
        for b in range(4):
            for j in range(int(c.cu[b + 1] - c.cu[b])):
                at, t = int(c.cached[b]) + j, int(c.cu[b]) + j
                bad = {p for p in (int(c.cached[b]) + first, 0)
                       if p < int(c.lens[b]) and at - 50 < p <= at}
                seen += bool(bad)
                if not bad:
                    assert bool(((out[t] - want[t]).abs() <= tol[t]).all()), f"row {t}, from {first}"
        assert seen > 0


@pytest.mark.parametrize("H", [1, 4])
def test_infinite_values_that_take_part(H):
    c = Case(8, [50, 20], [4, 1], 4 * H, H, 64, 16, lean=0.0)
    c.v[c.table[0, 3], 4, 0, 5] = math.inf  # position 52
    out = c.run().cpu().float()
    for j in range(4):
        assert bool((out[j, :4, 5] == math.inf).all()) == (j >= 2)
        assert torch.isfinite(out[j, :4][:, [d for d in range(64) if d != 5]]).all()
    assert torch.isfinite(out[:2]).all() and torch.isfinite(out[4:]).all()
    assert torch.isfinite(out[:, 4:]).all()


def test_logits_of_minus_infinity():
    c = Case(9, [30, 40], [2, 1], 4, 2, 64, 16, lean=0.0)
    c.q[:] = 0
    c.q[:, :, 0] = 1
    c.k[..., 0] = -math.inf
    lse = torch.zeros(3, 4, device=DEV)
    out = c.run(lse=lse)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_scales():
    Case(10, [700, 0, 64], [2, 1, 3], 8, 2, 128, 16, lean=4.0, scale=8.0).check("large logits")
    Case(11, [700, 0, 64], [2, 1, 3], 8, 2, 128, 16, FP8, lean=4.0, scale=-3.0).check("negative")
    Case(12, [700, 90], [2, 100], 8, 2, 128, 16, scale=-0.1).check("negative, many")


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own."""
    cases = [Case(13, [9000, 10, 3], [2, 1, 1], 8, 2, 128, 16), Case(14, [20, 900], [300, 5], 4, 2, 64, 16)]
    args = [(c.args(), c.kw()) for c in cases]
    want = [binding.attention_chunk_paged(*a, **k) for a, k in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(binding.attention_chunk_paged(*args[i][0], **args[i][1]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_graph_whose_requests_change():
    """A captured call replayed after requests came to have many rows, few, and
    none: which kernel reads a request is found on the device."""
    B, T = 6, 90
    c = Case(15, [300, 20, 64, 0, 9, 150], [15] * B, 8, 2, 128, 16)
    args, kw = c.args(), c.kw()
    out = torch.empty_like(args[0])
    n = binding.attention_chunk_workspace_bytes(T, B, 8, 2, 128, c.table.shape[1], 16)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    binding.attention_chunk_paged(*args, **kw, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.attention_chunk_paged(*args, **kw, out=out, workspace=ws)
    for new in ([15] * B, [1, 1, 1, 1, 1, 85 - 70], [0, 15, 2, 1, 0, 0], [0] * B, [15, 0, 15, 3, 1, 2]):
        c.cu = np.concatenate([[0], np.cumsum(new)])
        c.lens = c.cached + np.array(new)
        args[5].copy_(i32(c.lens))
        args[6].copy_(i32(c.cu))
        before = torch.full_like(c.q, 5.0)
        out.copy_(before)
        g.replay()
        torch.cuda.synchronize()
        want, _, tol, _ = c.want(before)
        assert bool(((out.cpu().double() - want).abs() <= tol).all()), str(new)


@pytest.mark.parametrize("Hq,H,D,bs,dtype", SHAPES)
def test_rows_behind_the_last_token(Hq, H, D, bs, dtype):
    """Requests of which only the first rows have a token in the cache: the
    others are zeros, whichever kernel reads the request."""
    for new in ([4, 1, 3, 2], [40, 7, 90, 1]):
        c = Case(16, [33, 0, 200, 64], new, Hq, H, D, bs, dtype)
        c.lens = c.cached + np.array([2, 0, 1 + new[2] // 3, 1])
        c.check(f"{new} {Hq}/{H}/{D}")


@pytest.mark.parametrize("new", [[1, 2, 1], [70, 3, 100]])
def test_scale_of_zero(new):
    """Every key that a row sees has the same weight."""
    c = Case(17, [300, 0, 64], new, 8, 2, 128, 16)
    c.scale = 0.0
    c.check("scale 0")


@pytest.mark.parametrize("B", [31, 32, 33])
def test_batches_around_the_number_of_both_kernels(B):
    """Many rows on average, few in most requests."""
    new = [1] * (B - 2) + [150, 200]
    rng = np.random.default_rng(B)
    Case(18, rng.integers(0, 200, B), new, 8, 2, 128, 16).check(f"{B} requests")


def test_requests_that_share_their_blocks():
    """Two rows of the table over the same blocks, one token apart."""
    c = Case(19, [100, 100, 100], [2, 1, 40], 8, 2, 64, 16)
    c.table[1] = c.table[0]
    c.table[2, :6] = c.table[0, :6]
    c.check("shared")


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("new", [[2, 1, 1], [2, 300, 40]])
def test_pools_past_32_bits(dtype, new):
    """Blocks whose elements and bytes lie past 2^32: the same bits as from a small
    pool; and the blocks moved there by a copy."""
    c = Case(20, [500, 0, 90], new, 8, 2, 128, 64, dtype)
    args, kw = c.args(), c.kw()
    want = binding.attention_chunk_paged(*args, **kw)
    n = c.k.shape[0]
    slot = 64 * 2 * 128
    nb = (1 << 32) // slot * (1 if dtype == BF16 else 2) + 1000
    big = [torch.full((nb, 64, 2, 128), math.nan, device=DEV, dtype=BF16).to(dtype)
           if dtype == BF16 else
           torch.full((nb, 64, 2, 128), 0x7f, device=DEV, dtype=torch.uint8).view(dtype)
           for _ in range(2)]
    for x, small in zip(big, args[1:3]):
        x.view(torch.uint8)[:n].copy_(small.view(torch.uint8))
    src, dst = np.arange(n), nb - 1 - 7 * np.arange(n)
    binding.paged_copy(i32(src), i32(dst), *big)
    table = np.where(c.table < 0, -1, nb - 1 - 7 * np.clip(c.table, 0, n - 1))
    got = binding.attention_chunk_paged(args[0], *big, i32(table), *args[4:], **kw)
    assert torch.equal(got, want)
