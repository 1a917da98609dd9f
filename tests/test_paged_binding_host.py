"""Sizes past 32 bits in the paged cache's binding (no GPU needed: the calls are
refused, or their arguments looked at in place of a launch)."""
import pytest
import torch

from mixture_value_projection_amd import binding

I32 = torch.int32
HUGE = [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63]


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.fixture
def launched(monkeypatch):
    """The arguments of each launch."""
    calls = []
    monkeypatch.setattr(binding, "_launch", lambda fn, name, device, *args: calls.append(args))
    return calls


def attend(window):
    q, pool = z(2, 4, 64), z(5, 16, 2, 64)
    binding.attention_paged(q, pool, pool, z(2, 3, dtype=I32), z(2, dtype=I32), 1.0, window=window)


@pytest.mark.parametrize("window", HUGE)
def test_window_wider_than_any_request(launched, window):
    """Such a window leaves nothing out, and is not cut to its lowest 32 bits."""
    attend(window)
    assert launched[0][18] == 2 ** 31 - 1
    attend(37)
    attend(-window)  # negative ones stay so, for the library to refuse
    assert launched[1][18] == 37 and launched[2][18] == -1


@pytest.mark.parametrize("n", HUGE)
def test_sizes_past_32_bits_are_refused(launched, n):
    table, lens, free, count = z(2, 3, dtype=I32), z(2, dtype=I32), z(9, dtype=I32), z(1, dtype=I32)
    for T, bs in [(n, 16), (4, n)]:
        with pytest.raises(ValueError):
            binding.paged_plan(lens, lens, T, bs, table, free, count)
    with pytest.raises(ValueError):
        binding.attention_workspace_bytes(2, 4, 2, 64, 3, 16, n)
    q, kb = z(2, 4, 64), z(5, 2, 2, 64)
    for bs, keep, first, last in [(n, 4, 1, 1), (16, n, 1, 1), (16, 4, n, 1), (16, 4, 1, n)]:
        with pytest.raises(ValueError):
            binding.block_select(q, kb, bs, table, lens, keep, first, last)
    assert not launched


def test_pools_of_more_blocks_than_32_bits_are_refused(launched):
    """A view of one row stands in for a pool of 2^32 + 5 blocks (its strides,
    too, are refused, but its blocks are counted first)."""
    row = z(1, 1, 1, 64).expand(2 ** 32 + 5, 1, 1, 64)
    k, slots = z(3, 1, 64), z(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="32 bits"):
        binding.kv_store_paged(k, None, row, None, slots)
    with pytest.raises(ValueError, match="32 bits"):
        binding.attention_paged(z(2, 4, 64), row, row, z(2, 3, dtype=I32), z(2, dtype=I32), 1.0)
    assert not launched
