"""The chunk attention writes nothing outside a workspace of the size that it asks
for, and what a workspace held before does not matter."""
import numpy as np
import pytest
import torch

from mixture_value_projection_amd import binding
from test_chunk_attention_gpu import BF16, DEV, FP8, Case

pytestmark = pytest.mark.gpu
GUARD = 1 << 20


@pytest.fixture(autouse=True)
def _gpu_only():
    assert torch.cuda.is_available(), "GPU test run without a GPU"
    binding.load_library()


def size_of(c, T=None):
    return binding.attention_chunk_workspace_bytes(T or c.q.shape[0], len(c.lens), c.q.shape[1],
                                                   c.k.shape[2], c.q.shape[2], c.table.shape[1], c.bs)


def guarded(c, n, fill):
    buf = torch.full((n + 2 * GUARD,), fill, dtype=torch.uint8, device=DEV)
    out = torch.zeros(c.q.shape, dtype=BF16, device=DEV)
    c.run(out=out, workspace=buf[GUARD:GUARD + n])
    assert bool((buf[:GUARD] == fill).all()) and bool((buf[GUARD + n:] == fill).all())
    return out


SPREAD = [int(3 * 900 ** ((0.31 + 0.618034 * i) % 1)) for i in range(70)]


@pytest.mark.parametrize("Hq,H,D,dtype", [(32, 8, 128, BF16), (6, 3, 64, FP8), (4, 2, 256, BF16),
                                          (17, 1, 64, BF16), (8, 4, 128, FP8), (16, 1, 256, FP8)])
@pytest.mark.parametrize("cached,new", [
    ([130], [1]), ([130], [19]), ([0], [700]), ([9000], [2]), ([9000], [40]),
    (SPREAD[:7], [1, 40, 3, 0, 130, 1, 64]), (SPREAD, [1] * 66 + [90, 5, 0, 200]),
    ([5000] * 3, [1, 2, 1]), ([0] * 40, [16] * 40),
])
def test_nothing_outside(Hq, H, D, dtype, cached, new):
    c = Case(1, cached, new, Hq, H, D, 16, dtype, padding=3)
    n = size_of(c)
    first = guarded(c, n, 0)
    for fill in (255, 77):
        assert torch.equal(first, guarded(c, n, fill))
    # In the workspace of a call of more tokens.
    assert torch.equal(first, guarded(c, size_of(c, 2000), 255))


def test_results_do_not_hang_on_the_width_of_the_table():
    """A wider table row asks for more workgroups; the lines of work are cut alike."""
    for cached, new in (([300, 20], [2, 1]), ([300, 20], [40, 9]), ([2000] * 9, [1] * 9)):
        a = Case(2, cached, new, 8, 2, 128, 16)
        b = Case(2, cached, new, 8, 2, 128, 16, width=6000)
        assert size_of(b) > size_of(a)
        assert torch.equal(a.run(), b.run())
