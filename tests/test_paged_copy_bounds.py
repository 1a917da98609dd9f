"""paged_copy of the key bounds alone, as the C call takes them (a cache whose
keys and values another tool moves)."""
import numpy as np
import pytest
import torch

from mixture_value_projection_amd import binding

I32 = torch.int32


class Launched(Exception):
    pass


def test_bounds_alone_reach_the_library(monkeypatch):
    """The call's arguments, with no GPU."""
    def launch(fn, what, dev, *args):
        raise Launched(args)
    monkeypatch.setattr(binding, "_launch", launch)
    pairs, bounds = torch.zeros(2, dtype=I32), torch.zeros(3, 2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(Launched) as got:
        binding.paged_copy(pairs, pairs, None, k_bounds=bounds)
    args = got.value.args[0]
    assert args[2] == 2 and args[4:6] == (None, None) and args[6] == bounds.data_ptr()
    assert args[7] == 0 and args[8] == 3 and args[9] > 0 and args[10:] == (2, 64)


@pytest.mark.parametrize("bounds", [
    None, torch.zeros(3, 2, 2, 64), torch.zeros(3, 2, 64, dtype=torch.bfloat16),
    torch.zeros(3, 2, 3, 64, dtype=torch.bfloat16),
    torch.zeros(3, 2, 2, 128, dtype=torch.bfloat16)[..., ::2],
    torch.zeros(3, 2, 2, 64, dtype=torch.bfloat16),  # not on a GPU
])
def test_other_bounds_are_refused(bounds):
    pairs = torch.zeros(2, dtype=I32)
    with pytest.raises(ValueError):
        binding.paged_copy(pairs, pairs, None, k_bounds=bounds)


@pytest.mark.gpu
@pytest.mark.parametrize("H,D", [(8, 128), (1, 16), (3, 64)])
def test_bounds_alone(H, D):
    g = torch.Generator().manual_seed(H)
    nb = 30
    bounds = torch.randn(nb, H, 2, D, generator=g).to(torch.bfloat16)
    perm = np.random.default_rng(H).permutation(nb)
    src, dst = perm[:10].copy(), perm[10:20].copy()
    src[2], dst[4] = -1, nb
    want = bounds.clone()
    for s, d in zip(src, dst):
        if s >= 0 and d < nb:
            want[d] = bounds[s]
    got = bounds.cuda()
    binding.paged_copy(*(torch.as_tensor(x.astype(np.int32)).cuda() for x in (src, dst)), None,
                       k_bounds=got)
    assert torch.equal(got.cpu(), want)
