"""The key bounds of blocks through a fork, stores behind it, a cut, a compaction
and stores behind that: those of the keys that the requests hold there."""
import numpy as np
import pytest
import torch

from mixture_value_projection_amd import binding
import blockslib as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP8 = torch.bfloat16, R.FP8


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device=DEV)


@pytest.mark.parametrize("dtype,bs,H,D", [(BF16, 16, 2, 64), (FP8, 24, 3, 128), (BF16, 1, 1, 256)])
def test_bounds_follow_the_blocks(dtype, bs, H, D):
    assert torch.cuda.is_available(), "GPU test run without a GPU"
    g = torch.Generator(device=DEV).manual_seed(1)
    B, mb, nb = 8, 160, 400
    k_cache = torch.full((nb, bs, H, D), float("nan"), device=DEV).to(dtype)
    v_cache = k_cache.clone()
    bounds = torch.full((nb, H, 2, D), float("nan"), dtype=BF16, device=DEV)
    table = torch.full((B, mb), -1, dtype=torch.int32, device=DEV)
    free, count = i32(np.random.default_rng(0).permutation(nb)), i32([nb])
    shares = torch.zeros(nb, dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    keys = [torch.zeros(0, H, D) for _ in range(B)]

    def step(new):
        nonlocal lens, count
        p = binding.paged_plan(lens, i32(new), sum(new), bs, table, free, count)
        k = torch.randn(sum(new), H, D, generator=g, device=DEV).to(BF16)
        binding.kv_store_paged(k, k, k_cache, v_cache, p.slot_mapping, k_bounds=bounds)
        rows = k.to(dtype).float().cpu() if dtype == FP8 else k.float().cpu()
        at = 0
        for b, n in enumerate(new):
            keys[b] = torch.cat([keys[b], rows[at:at + n]])
            at += n
        lens, count = p.seq_lens, p.free_count

    def check(what):
        """Bounds, and the blocks chosen by them, against the requests' own keys."""
        got, t = bounds.float().cpu(), table.cpu().numpy()
        assert lens.tolist() == [len(x) for x in keys], what
        for b, x in enumerate(keys):
            for j in range(R.ceil_div(len(x), bs)):
                mine = x[j * bs:(j + 1) * bs]
                want = torch.stack([mine.amin(0), mine.amax(0)], 1)
                assert torch.equal(got[t[b, j]], want), f"{what}: block {j} of request {b}"
        q = torch.randn(B, 2 * H, D, generator=g, device=DEV).to(BF16)
        keep = 5
        sel = binding.block_select(q, bounds, bs, table, lens, keep=keep).cpu().numpy()
        for b, x in enumerate(keys):
            n = R.ceil_div(len(x), bs)
            for h in range(H):
                score = []
                for j in range(n):
                    mine = x[j * bs:(j + 1) * bs, h].double()
                    lo, hi = mine.amin(0), mine.amax(0)
                    two = q[b, 2 * h:2 * h + 2].cpu().double()
                    score.append(float(torch.where(two > 0, hi * two, lo * two).sum(1).max()))
                # (The first and the last block are always in.)
                want = sorted(sorted(range(n), key=lambda j: (j not in (0, n - 1), -score[j], j))[:keep])
                assert [j for j in sel[b, h].tolist() if j >= 0] == want, f"{what}: choice {b} {h}"

    step([100, 37, 64, 0, 0, 0, 0, 0])
    check("prompts")
    f = binding.paged_fork(i32([0, 1, 2, 0]), i32([3, 4, 5, 6]), bs, table, lens, free, count, shares,
                           fork_lens=i32([100, 37, 64, 50]))
    binding.paged_copy(f.copy_src, f.copy_dst, k_cache, v_cache, k_bounds=bounds)
    lens, count = f.seq_lens, f.free_count
    for p, c, n in zip([0, 1, 2, 0], [3, 4, 5, 6], [100, 37, 64, 50]):
        keys[c] = keys[p][:n].clone()
    step([3, 1, 2, 1, 9, 3, 1, 0])  # (row 6 begins inside one of its parent's blocks)
    check("forked")
    r = binding.paged_free(lens, i32([0, 37, 0, 101, 44, 66, 51, 0]), bs, table, free, count, shares)
    lens, count = r.seq_lens, r.free_count
    for b, n in enumerate([0, 37, 0, 101, 44, 66, 51, 0]):
        keys[b] = keys[b][:n]
    step([0, 2, 0, 1, 3, 1, 2, 20])
    check("cut")
    c = binding.paged_compact(lens, bs, table, free, count, shares)
    binding.paged_copy(c.move_src, c.move_dst, k_cache, v_cache, k_bounds=bounds, count=c.move_count)
    count = c.free_count
    assert int(c.move_count) > 0
    check("moved")
    step([30, 1, 1, 2, 1, 3, 1, 1])
    check("stored behind the move")
