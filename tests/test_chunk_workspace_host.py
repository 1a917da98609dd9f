"""Sizes of the chunk attention's workspace (CPU only): by what a call can need,
not by the largest, and never less for a larger call."""
import random

import pytest

from mixture_value_projection_amd import binding

size = binding.attention_chunk_workspace_bytes


def parts(D, floats):
    """Bytes of so many parts of a row: its channels, maximum and sum."""
    return 4 * floats * (D + 2)


@pytest.mark.parametrize("D,Hq,H", [(64, 4, 1), (64, 32, 8), (128, 32, 8), (256, 16, 4)])
def test_small_calls(D, Hq, H):
    # A token after 130 and 19 tokens after 130: a few stretches of the line of work.
    assert size(1, 1, Hq, H, D, 10, 16) <= 2 << 20
    assert size(19, 1, Hq, H, D, 10, 16) <= 8 << 20
    # A token after any length: the parts of few rows alone, of 16 rows and four key heads
    # from two tiles of each of 512 workgroups (256 where rows have 256 channels).
    groups = 256 if D == 256 else 512
    assert size(1, 1, Hq, H, D, 65536, 16) <= parts(D, groups * 2 * 64) + (64 << 10)


def test_no_parts_of_few_rows_for_wide_groups():
    # 256 rows from two tiles of each of 256 workgroups, and records.
    assert size(4096, 64, 32, 1, 128, 4096, 16) <= parts(128, 256 * 2 * 256) + (64 << 10)


def test_a_larger_call_has_the_room_of_a_smaller_one():
    rng = random.Random(1)
    for _ in range(20000):
        D = rng.choice([64, 128, 256])
        H = rng.choice([1, 2, 3, 4, 8])
        Hq = H * rng.choice([1, 2, 3, 4, 5, 16, 17, 30])
        T, B = int(2 ** rng.uniform(0, 20)), int(2 ** rng.uniform(0, 11))
        bs = rng.choice([1, 8, 16, 24, 128])
        mb = int(2 ** rng.uniform(0, 14))
        n = size(T, B, Hq, H, D, mb, bs)
        t, b, m = (rng.randint(1, T), rng.randint(1, B), rng.randint(1, mb))
        assert size(t, b, Hq, H, D, m, bs) <= n, (T, B, Hq, H, D, mb, bs, t, b, m)
        assert n % 256 == 0 and n <= parts(D, 512 * 2 * 64 + 256 * 2 * 256) + (64 << 10)
