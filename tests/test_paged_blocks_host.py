"""Host-side refusals of the chunk attention and the block upkeep: every call
here returns from the argument checks (or has nothing to do), so no kernel is
launched and no GPU is needed."""
import ctypes
import os

import pytest
import torch

from mixture_value_projection_amd import binding
from mixture_value_projection_amd.build import LIBPATH

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
FAKE = 1 << 20  # an aligned non-null address that is never dereferenced
BAD = ctypes.c_size_t(-1).value
I32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIBPATH):
        pytest.fail(f"{LIBPATH} not built (run __graft_entry__.build())")
    return binding.load_library()


def call(fn, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return fn(*a.values())


CHUNK = dict(q=FAKE, k=FAKE, v=FAKE, dtype=1, ks=FAKE, vs=FAKE, nb=40, bs=16, table=FAKE, mb=10,
             cached=FAKE, lens=FAKE, cu=FAKE, T=8, B=4, Hq=32, H=8, D=128, scale=0.1, window=0,
             out=FAKE + 4096, lse=FAKE, ws=FAKE, wsb=1 << 40, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(mb=0), INVALID), (dict(bs=0), INVALID),
    (dict(nb=-1), INVALID), (dict(Hq=0), INVALID), (dict(H=0), INVALID), (dict(D=0), INVALID),
    (dict(window=-1), INVALID), (dict(dtype=2), INVALID), (dict(dtype=0), INVALID),
    (dict(T=(1 << 24) + 1), UNSUPPORTED), (dict(B=2049), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(Hq=33), UNSUPPORTED), (dict(H=256, Hq=256), UNSUPPORTED), (dict(Hq=2048), UNSUPPORTED),
    (dict(mb=1 << 27), UNSUPPORTED), (dict(nb=1 << 28), UNSUPPORTED),
    (dict(T=1 << 20, mb=1 << 24, bs=16), UNSUPPORTED),  # 2^20 rows of 32 heads over 2^28 keys
    (dict(scale=float("nan")), UNSUPPORTED), (dict(scale=float("inf")), UNSUPPORTED),
    *[({n: None}, INVALID) for n in ("q", "k", "v", "table", "cached", "lens", "cu", "out")],
    *[({n: FAKE + 8}, INVALID) for n in ("q", "k", "v", "out")],
    (dict(out=FAKE), INVALID),
    *[({n: FAKE + 2}, INVALID) for n in ("ks", "vs", "table", "cached", "lens", "cu", "lse")],
    (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE), (dict(ws=FAKE + 16), INVALID),
    (dict(T=0, q=None, ws=None), OK), (dict(B=0, table=None, ws=None), OK),
])
def test_chunk_rejects(lib, kw, rc):
    assert call(lib.mova_attention_chunk_paged, CHUNK, kw) == rc


def test_chunk_workspace(lib):
    size = lib.mova_attention_chunk_workspace_bytes
    assert size(8, 4, 33, 8, 128, 10, 16) == BAD and size(8, 4, 32, 8, 96, 10, 16) == BAD
    assert size(1 << 24, 2048, 1024, 1, 128, 10, 16) != BAD
    with pytest.raises(binding.MovaError):
        binding.attention_chunk_workspace_bytes(8, 4, 33, 8, 128, 10, 16)


FORK = dict(par=FAKE, chi=FAKE, take=None, n=3, cached=FAKE, B=4, bs=16, mb=10, table=FAKE, free=FAKE,
            cap=40, count=FAKE, count_out=FAKE + 4, shares=FAKE, nb=40, seq=FAKE + 64, src=FAKE,
            dst=FAKE + 128, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(n=-1), INVALID), (dict(B=-1), INVALID), (dict(bs=0), INVALID), (dict(mb=0), INVALID),
    (dict(cap=-1), INVALID), (dict(nb=-1), INVALID), (dict(n=2049), UNSUPPORTED),
    (dict(B=2049), UNSUPPORTED), (dict(mb=1 << 27), UNSUPPORTED),
    (dict(nb=(1 << 20) + 1), UNSUPPORTED),
    *[({n: None}, INVALID) for n in ("par", "chi", "cached", "table", "free", "count", "count_out",
                                     "shares", "seq", "src", "dst")],
    *[({n: FAKE + 2}, INVALID) for n in ("par", "chi", "take", "cached", "table", "free", "count",
                                         "count_out", "shares", "seq", "src", "dst")],
    (dict(count_out=FAKE), INVALID), (dict(seq=FAKE), INVALID), (dict(dst=FAKE), INVALID),
    (dict(take=FAKE + 64), INVALID),
])
def test_fork_rejects(lib, kw, rc):
    assert call(lib.mova_paged_fork, FORK, kw) == rc


FREE = dict(cached=FAKE, keep=FAKE, B=4, bs=16, mb=10, table=FAKE, free=FAKE, cap=40, count=FAKE,
            count_out=FAKE + 4, shares=FAKE, nb=40, seq=FAKE + 64, ws=FAKE, wsb=1 << 20,
            stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), INVALID), (dict(bs=0), INVALID), (dict(mb=0), INVALID), (dict(cap=-1), INVALID),
    (dict(nb=-1), INVALID), (dict(B=2049), UNSUPPORTED), (dict(mb=1 << 27), UNSUPPORTED),
    (dict(nb=(1 << 20) + 1), UNSUPPORTED),
    *[({n: None}, INVALID) for n in ("cached", "keep", "table", "free", "count", "count_out",
                                     "shares", "seq")],
    *[({n: FAKE + 2}, INVALID) for n in ("cached", "keep", "table", "free", "count", "count_out",
                                         "shares", "seq")],
    (dict(count_out=FAKE), INVALID), (dict(seq=FAKE), INVALID),
    (dict(keep=FAKE + 64), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=8), WORKSPACE), (dict(ws=FAKE + 16), INVALID),
])
def test_free_rejects(lib, kw, rc):
    assert call(lib.mova_paged_free, FREE, kw) == rc


COMPACT = dict(cached=FAKE, B=4, bs=16, mb=10, table=FAKE, table_out=FAKE, free=FAKE, free_out=FAKE,
               cap=40, count=FAKE, count_out=FAKE + 4, shares=FAKE, shares_out=FAKE, nb=40, limit=0,
               remap=FAKE, src=FAKE, dst=FAKE, moves=FAKE, ws=FAKE, wsb=1 << 20, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), INVALID), (dict(bs=0), INVALID), (dict(mb=0), INVALID), (dict(cap=-1), INVALID),
    (dict(nb=-1), INVALID), (dict(limit=-1), INVALID), (dict(B=2049), UNSUPPORTED),
    (dict(mb=1 << 27), UNSUPPORTED), (dict(nb=(1 << 20) + 1), UNSUPPORTED),
    *[({n: None}, INVALID) for n in ("cached", "table", "table_out", "free", "free_out", "count",
                                     "count_out", "shares", "shares_out", "remap", "src", "dst",
                                     "moves")],
    *[({n: FAKE + 2}, INVALID) for n in ("cached", "table", "table_out", "free", "free_out", "count",
                                         "count_out", "shares", "shares_out", "remap", "src", "dst",
                                         "moves")],
    (dict(count_out=FAKE), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=8), WORKSPACE), (dict(ws=FAKE + 16), INVALID),
])
def test_compact_rejects(lib, kw, rc):
    assert call(lib.mova_paged_compact, COMPACT, kw) == rc


def test_free_workspace(lib):
    size = lib.mova_paged_free_workspace_bytes
    assert size(-1) == BAD and size((1 << 20) + 1) == BAD
    for nb in (0, 1, 1024, 1025, 262144, 262145, 1 << 20):
        # A count of each of 256 runs, and 16 bits a block in whole words.
        assert size(nb) >= 4 * 256 + 4 * ((nb + 1) // 2) and size(nb) % 256 == 0


def test_compact_workspace(lib):
    size = lib.mova_paged_compact_workspace_bytes
    assert size(-1) == BAD and size((1 << 20) + 1) == BAD
    for nb in (0, 1, 255, 256, 257, 1 << 20):
        # A count a run of 256 blocks, one more, and a bit a block of whole runs.
        runs = -(-nb // 256)
        assert size(nb) >= 4 * (runs + 1) + 32 * runs and size(nb) % 256 == 0


COPY = dict(src=FAKE, dst=FAKE, n=3, count=FAKE, k=FAKE, v=FAKE, kb=FAKE, dtype=1, nb=40, bs=16, H=8,
            D=128, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(n=-1), INVALID), (dict(nb=-1), INVALID), (dict(bs=0), INVALID), (dict(H=0), INVALID),
    (dict(D=0), INVALID), (dict(D=72), UNSUPPORTED), (dict(H=129), UNSUPPORTED),
    (dict(nb=(1 << 31) - 1, bs=1024), UNSUPPORTED), (dict(bs=(1 << 18) + 1), UNSUPPORTED),
    (dict(dtype=2), INVALID), (dict(src=None), INVALID), (dict(dst=None), INVALID),
    (dict(k=None, v=None, kb=None), INVALID),
    *[({n: FAKE + 2}, INVALID) for n in ("src", "dst", "count")],
    *[({n: FAKE + 8}, INVALID) for n in ("k", "v", "kb")],
    (dict(n=0, src=None), OK),
])
def test_copy_rejects(lib, kw, rc):
    assert call(lib.mova_paged_copy, COPY, kw) == rc


# ---- the binding ------------------------------------------------------------------

def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def chunk_args(**kw):
    a = dict(q=z(5, 4, 64), k_cache=z(3, 16, 2, 64), v_cache=z(3, 16, 2, 64),
             block_table=z(2, 3, dtype=I32), cached_lens=z(2, dtype=I32), seq_lens=z(2, dtype=I32),
             cu_new=z(3, dtype=I32), scale=1.0)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw", [
    dict(q=z(5, 4, 64, dtype=torch.float32)), dict(q=z(5, 256)), dict(q=z(5, 4, 128)[:, :, ::2]),
    dict(v_cache=z(3, 16, 2, 64).to(torch.float8_e4m3fn)), dict(v_cache=z(4, 16, 2, 64)),
    dict(k_cache=z(3, 16, 2, 128)), dict(block_table=z(2, 3, dtype=torch.int64)),
    dict(cached_lens=z(3, dtype=I32)), dict(seq_lens=z(1, dtype=I32)), dict(cu_new=z(2, dtype=I32)),
    dict(k_scale=z(2)), dict(out=z(4, 4, 64)), dict(lse=z(5, 4)),
    dict(workspace=z(9, dtype=torch.float32)),
    {},  # not on a GPU
])
def test_chunk_binding_refuses(kw):
    with pytest.raises(ValueError):
        binding.attention_chunk_paged(**chunk_args(**kw))


def upkeep(**kw):
    a = dict(block_size=16, block_table=z(4, 3, dtype=I32), cached_lens=z(4, dtype=I32),
             free_blocks=z(9, dtype=I32), free_count=z(1, dtype=I32), shares=z(9, dtype=I32))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw", [
    dict(block_table=z(4, 3, dtype=torch.int64)), dict(block_table=z(12, dtype=I32)),
    dict(cached_lens=z(3, dtype=I32)), dict(free_blocks=z(9, 1, dtype=I32)),
    dict(free_count=z(2, dtype=I32)), dict(shares=z(9)), dict(block_size=2 ** 31),
    dict(block_size=2 ** 32 + 16), {},
])
def test_upkeep_bindings_refuse(kw):
    pairs = z(2, dtype=I32)
    with pytest.raises(ValueError):
        binding.paged_fork(pairs, pairs, **upkeep(**kw))
    with pytest.raises(ValueError):
        binding.paged_free(keep_lens=z(4, dtype=I32), **upkeep(**kw))
    with pytest.raises(ValueError):
        binding.paged_compact(**upkeep(**kw))


def test_more_bindings_refuse():
    pairs = z(2, dtype=I32)
    for kw in (dict(children=z(3, dtype=I32)), dict(fork_lens=z(3, dtype=I32)),
               dict(copy_src=z(3, dtype=I32)), dict(seq_lens=z(3, dtype=I32))):
        with pytest.raises(ValueError):
            binding.paged_fork(**{**dict(parents=pairs, children=pairs), **upkeep(), **kw})
    with pytest.raises(ValueError):
        binding.paged_free(keep_lens=z(3, dtype=I32), **upkeep())
    for kw in (dict(limit=2 ** 31), dict(remap=z(8, dtype=I32)), dict(move_src=z(9, dtype=I32)),
               dict(shares_out=z(8, dtype=I32)), dict(block_table_out=z(4, 2, dtype=I32))):
        with pytest.raises(ValueError):
            binding.paged_compact(**upkeep(**kw))
    pool = z(3, 16, 2, 64)
    for args, kw in [((pairs, pairs, None), {}), ((pairs, z(3, dtype=I32), pool), {}),
                     ((pairs, pairs, pool, z(3, 16, 2, 128)), {}),
                     ((pairs, pairs, pool), dict(k_bounds=z(3, 2, 2, 32))),
                     ((pairs, pairs, pool), dict(count=z(2, dtype=I32))),
                     ((pairs, pairs, pool, pool.to(torch.float8_e4m3fn)), {}),
                     ((pairs, pairs, pool), {})]:
        with pytest.raises(ValueError):
            binding.paged_copy(*args, **kw)
