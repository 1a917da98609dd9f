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
