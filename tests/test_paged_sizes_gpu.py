"""Calls of the paged cache's operators above the sizes where their kernels go
over their work more than once."""
import numpy as np
import pytest
import torch

from mixture_value_projection_amd import binding
import pagedlib as R
import test_paged_cache_gpu as C

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_only():
    assert torch.cuda.is_available(), "GPU test run without a GPU"
    binding.load_library()


@pytest.mark.parametrize("with_bounds", [False, True])
def test_store_most_tokens(with_bounds):
    """2^24 rows of 1552 elements (48.5 GiB, most of them without a slot): with a
    wave for each of a row's four pieces the launch would have 2^32 threads, one
    more than is allowed."""
    T, H, D, bs, nb = 1 << 24, 97, 16, 4, 40
    k = torch.empty(T, H, D, dtype=torch.bfloat16, device=C.DEV)
    slots = torch.full((T,), -1, dtype=torch.int64, device=C.DEV)
    # Whole and partly filled blocks at the beginning, in the middle and at the end.
    rows = np.concatenate([np.arange(10), np.arange(10) + T // 2 - 5, np.arange(10) + T - 10])
    at = np.concatenate([np.arange(10) + 8, np.arange(10) + 40, np.arange(10) + 100])
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(len(rows), H, D, generator=gen).to(torch.bfloat16)
    k[rows.tolist()] = x.to(C.DEV)
    slots[rows.tolist()] = torch.from_numpy(at).to(C.DEV)
    pool = torch.randn(nb, bs, H, D, generator=gen).to(torch.bfloat16)
    before = torch.full((nb, H, 2, D), 7.0, dtype=torch.bfloat16)
    got, kb = pool.to(C.DEV), before.to(C.DEV)
    binding.kv_store_paged(k, None, got, None, slots, k_bounds=kb if with_bounds else None)
    torch.cuda.synchronize()
    want = R.store(x, pool, at, None)
    assert torch.equal(got.cpu(), want)
    if with_bounds:
        before = R.bounds(want, at, before)
    assert torch.equal(kb.cpu(), before)


@pytest.mark.parametrize("seed,kw", [
    (1, dict(B=40, bs=16, mb=700, longest=900, most_new=6000, ended=3)),
    (2, dict(B=2048, bs=8, mb=64, longest=300, most_new=150, ended=200, short=700, extra_rows=3)),
    (5, dict(B=1, bs=4, mb=40000, longest=50, most_new=150000)),
])
def test_plan_many_tokens(seed, kw):
    """More token rows than the launch has threads (128 workgroups of 256)."""
    case = C.plan_case(seed, **kw)
    assert case[2] > 32768, case[2]
    C.check_plan(*case, what=str(kw))


def test_plan_many_blocks_back():
    """Two thirds of a million blocks given back, and many of them handed out, by one
    call."""
    B, bs, mb = 300, 1, 4000
    rng = np.random.default_rng(4)
    cached = rng.integers(2500, mb + 1, B)
    new = np.full(B, -1)
    new[::3], cached[::3] = rng.integers(1000, 3000, B)[::3], 0
    held = int(cached.sum())
    table = np.full((B, mb), -1)
    perm, at = rng.permutation(held), 0
    for b in range(B):
        table[b, :cached[b]] = perm[at:at + cached[b]]
        at += cached[b]
    C.check_plan(cached, new, int(new.clip(0).sum()), bs, table, np.full(held, -1), 0, "back")


@pytest.mark.parametrize("dtype", [torch.bfloat16, C.FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T,most,bs", [(17000, 1, 4), (20000, 40, 16), (40000, 9, 8)])
def test_store_many_tokens(T, most, bs, dtype):
    """Several runs among the up to 64 tokens whose bounds one workgroup forms."""
    rng = np.random.default_rng(T)
    H, D = 2, 16
    nb = T
    pages, slots = iter(rng.permutation(nb)), []
    while len(slots) < T - most - 1:
        at = next(pages) * bs + rng.integers(bs)
        for i in range(rng.integers(1, most + 1)):
            if i and at % bs == 0:  # the block is full
                at = next(pages) * bs
            slots.append(at)
            at += 1
        if len(slots) % 50 < 2:
            slots.append(rng.choice([-1, nb * bs]))  # rows without a slot between runs
    slots = np.array(slots + [-1] * (T - len(slots)), dtype=np.int64)
    pool = C.make_pool(rng, nb, bs, H, D, dtype)
    x = torch.from_numpy(rng.standard_normal((T, H, D), dtype=np.float32) * 3).to(torch.bfloat16)
    scale = torch.tensor([0.02, 0.013]) if dtype == C.FP8 else None
    before = torch.full((nb, H, 2, D), 7.0, dtype=torch.bfloat16)
    got, kb = pool.to(C.DEV), before.to(C.DEV)
    binding.kv_store_paged(x.to(C.DEV), None, got, None, torch.as_tensor(slots, device=C.DEV),
                           k_scale=None if scale is None else scale.to(C.DEV), k_bounds=kb)
    torch.cuda.synchronize()
    want = R.store(x, pool, slots, scale)
    assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))
    assert torch.equal(kb.cpu(), R.bounds(want, slots, before))


@pytest.mark.parametrize("n,keep,first,last", [(65537, 1100, 1, 1), (70000, 1200, 0, 3),
                                               (131000, 20, 2, 2)])
def test_select_over_more_than_65536_blocks(n, keep, first, last):
    """Lists of more blocks than have a mark in LDS; with few wanted only the
    promising tiles of them are looked at."""
    rng = np.random.default_rng(n)
    H, D, G = 1, 64, 2
    nb, bs = n + 5, 2
    lens = [2 * n - 1, 77]
    table = np.stack([rng.permutation(nb)[:n + 3] for _ in lens])
    q = torch.from_numpy(rng.standard_normal((2, H * G, D), dtype=np.float32)).to(torch.bfloat16)
    kb = torch.sort(torch.from_numpy(rng.standard_normal((nb, H, 2, D), dtype=np.float32)),
                    dim=2).values.to(torch.bfloat16)
    C.check_select(q, kb, bs, table, lens, keep, first, last, "random")
    qi = torch.from_numpy(rng.integers(-1, 2, q.shape)).to(torch.bfloat16)
    ki = torch.from_numpy(rng.integers(-1, 2, kb.shape)).to(torch.bfloat16)
    C.check_select(qi, ki, bs, table, lens, keep, first, last, "ties")
    holes = table.copy()
    holes[:, ::3] = -1
    C.check_select(q, kb, bs, holes, lens, keep, first, last, "holes")


@pytest.mark.parametrize("dtype", [torch.bfloat16, C.FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("B,Hq,H,D,bs,longest", [
    (300, 4, 2, 64, 8, 768), (300, 4, 2, 64, 8, 776), (180, 12, 4, 128, 16, 512),
    (180, 12, 4, 128, 16, 528), (90, 8, 4, 256, 16, 256), (90, 8, 4, 256, 16, 272)])
def test_more_rows_than_workgroups(B, Hq, H, D, bs, longest, dtype):
    """Batches of more rows than have a workgroup at once, on either side of the
    length (of bf16 keys) up to which each is one workgroup's."""
    rng = np.random.default_rng(longest)
    lens = rng.integers(0, longest + 1, B)
    lens[B // 2] = longest
    C.check_attention(C.make_attention(B, list(lens), Hq, H, D, bs, dtype), "more rows")
