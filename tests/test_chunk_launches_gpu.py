"""How many kernels a call of the chunk attention launches, counted in a captured
graph, and its results in batches around the rule that decides it."""
import ctypes

import numpy as np
import pytest
import torch

from mixture_value_projection_amd import binding
from test_chunk_attention_gpu import BF16, FP8, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_only():
    assert torch.cuda.is_available(), "GPU test run without a GPU"
    binding.load_library()


def launches(c):
    args, kw = c.args(), c.kw()
    out = torch.empty_like(args[0])
    T, Hq, D = c.q.shape
    ws = torch.empty(binding.attention_chunk_workspace_bytes(T, len(c.lens), Hq, c.k.shape[2], D,
                                                             c.table.shape[1], c.bs),
                     dtype=torch.uint8, device=out.device)
    binding.attention_chunk_paged(*args, **kw, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        binding.attention_chunk_paged(*args, **kw, out=out, workspace=ws)
    n = ctypes.c_size_t(0)
    hip = binding.load_library()  # (whose symbols are found with those of what it links)
    assert hip.hipGraphGetNodes(ctypes.c_void_p(g.raw_cuda_graph()), None, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("Hq,H,want", [
    (17, 1, 2), (40, 2, 2), (16, 1, 3), (8, 2, 3),
])
@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_groups_wider_than_the_few_rows(Hq, H, want, dtype):
    """Requests whose single tokens have more rows than the few-rows kernel takes
    are not looked for by it."""
    rng = np.random.default_rng(Hq)
    new = rng.integers(0, 3, 40)
    new[[3, 20]] = 30
    c = Case(1, rng.integers(0, 300, 40), new, Hq, H, 64, 16, dtype, refused=[5, 20], padding=4)
    c.check(f"40 requests, {Hq} heads over {H}")
    assert launches(c) == want


@pytest.mark.parametrize("new,want", [([1, 1, 1, 1], 2), ([4], 2), ([5], 2), ([2, 9, 1, 1], 3), ([300], 2)])
def test_launches_of_small_batches(new, want):
    c = Case(2, [70] * len(new), new, 8, 2, 128, 16)
    c.check(str(new))
    assert launches(c) == want
