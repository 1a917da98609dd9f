"""Host-side refusals of the paged cache's entry points: every call here
returns from the argument checks (or has nothing to do), so no kernel is
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


PLAN = dict(cached=FAKE, new=FAKE, B=4, T=8, bs=16, mb=10, table=FAKE, free=FAKE, cap=40, count=FAKE,
            count_out=FAKE + 4, seq=FAKE + 64, cu=FAKE, slots=FAKE, pos=FAKE, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(bs=0), INVALID), (dict(mb=0), INVALID),
    (dict(cap=-1), INVALID), (dict(B=2049), UNSUPPORTED), (dict(T=(1 << 24) + 1), UNSUPPORTED),
    (dict(mb=1 << 27), UNSUPPORTED),
    *[({n: None}, INVALID) for n in ("cached", "new", "table", "free", "count", "count_out", "seq",
                                     "cu", "slots", "pos")],
    *[({n: FAKE + 2}, INVALID) for n in ("cached", "new", "table", "free", "count", "count_out",
                                         "seq", "cu", "pos")],
    (dict(slots=FAKE + 4), INVALID),
    (dict(count_out=FAKE), INVALID), (dict(seq=FAKE), INVALID),
    (dict(seq=FAKE + 128, new=FAKE + 128), INVALID),
    (dict(B=0, count=None), INVALID),
])
def test_plan_rejects(lib, kw, rc):
    assert call(lib.mova_paged_plan, PLAN, kw) == rc


STORE = dict(k=FAKE, v=FAKE, T=8, H=8, D=128, kc=FAKE, vc=FAKE, dtype=1, ks=FAKE, vs=FAKE, nb=10,
             bs=16, slots=FAKE, kb=FAKE, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(D=0), INVALID), (dict(nb=-1), INVALID),
    (dict(bs=0), INVALID), (dict(D=72), UNSUPPORTED), (dict(H=129), UNSUPPORTED),
    (dict(T=(1 << 24) + 1), UNSUPPORTED), (dict(nb=(1 << 31) - 1, bs=1024), UNSUPPORTED),
    (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID), (dict(dtype=0), INVALID),
    (dict(ks=FAKE + 2), INVALID), (dict(k=None), INVALID), (dict(kc=None), INVALID),
    (dict(v=None), INVALID), (dict(vc=None), INVALID), (dict(slots=None), INVALID),
    (dict(k=None, kc=None), INVALID),                            # bounds without keys
    (dict(k=None, kc=None, v=None, vc=None, kb=None), INVALID),
    (dict(k=FAKE + 8), INVALID), (dict(vc=FAKE + 8), INVALID), (dict(kb=FAKE + 8), INVALID),
    (dict(slots=FAKE + 4), INVALID), (dict(T=0, k=None, slots=None), OK),
])
def test_store_rejects(lib, kw, rc):
    assert call(lib.mova_kv_store_paged, STORE, kw) == rc


SELECT = dict(q=FAKE, kb=FAKE, nb=40, bs=16, table=FAKE, mb=10, lens=FAKE, B=4, Hq=32, H=8, D=128,
              keep=8, first=1, last=2, sel=FAKE, ws=FAKE, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), INVALID), (dict(mb=0), INVALID), (dict(bs=0), INVALID), (dict(nb=-1), INVALID),
    (dict(Hq=0), INVALID), (dict(H=0), INVALID), (dict(D=0), INVALID), (dict(keep=0), INVALID),
    (dict(keep=-1), INVALID), (dict(first=-1), INVALID), (dict(last=-1), INVALID),
    (dict(first=7), INVALID), (dict(first=0, last=9), INVALID), (dict(B=2049), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED), (dict(Hq=33), UNSUPPORTED), (dict(H=256, Hq=256), UNSUPPORTED),
    (dict(Hq=2048), UNSUPPORTED), (dict(mb=1 << 27), UNSUPPORTED),
    (dict(keep=(1 << 20) + 1), UNSUPPORTED), (dict(nb=1 << 28), UNSUPPORTED),
    *[({n: None}, INVALID) for n in ("q", "kb", "table", "lens", "sel")],
    (dict(q=FAKE + 8), INVALID), (dict(kb=FAKE + 8), INVALID), (dict(table=FAKE + 2), INVALID),
    (dict(lens=FAKE + 2), INVALID), (dict(sel=FAKE + 2), INVALID), (dict(ws=None), WORKSPACE),
    (dict(wsb=100), WORKSPACE), (dict(ws=FAKE + 16), INVALID), (dict(B=0, q=None, ws=None), OK),
])
def test_select_rejects(lib, kw, rc):
    assert call(lib.mova_block_select, SELECT, kw) == rc


ATTEND = dict(q=FAKE, kc=FAKE, vc=FAKE, dtype=1, ks=FAKE, vs=FAKE, nb=40, bs=16, table=FAKE, mb=10,
              lens=FAKE, sel=FAKE, keep=4, B=4, Hq=32, H=8, D=128, scale=0.1, window=0, out=FAKE,
              lse=FAKE, ws=FAKE, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), INVALID), (dict(mb=0), INVALID), (dict(bs=0), INVALID), (dict(nb=-1), INVALID),
    (dict(Hq=0), INVALID), (dict(H=0), INVALID), (dict(D=0), INVALID), (dict(keep=-1), INVALID),
    (dict(keep=0), INVALID), (dict(sel=None), INVALID), (dict(window=-1), INVALID),
    (dict(dtype=2), INVALID), (dict(dtype=0), INVALID), (dict(ks=FAKE + 2), INVALID),
    (dict(B=2049), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(Hq=33), UNSUPPORTED),
    (dict(Hq=2048), UNSUPPORTED), (dict(mb=1 << 27), UNSUPPORTED), (dict(nb=1 << 28), UNSUPPORTED),
    (dict(keep=1 << 27), UNSUPPORTED), (dict(scale=float("nan")), UNSUPPORTED),
    (dict(scale=float("inf")), UNSUPPORTED),
    *[({n: None}, INVALID) for n in ("q", "kc", "vc", "table", "lens", "out")],
    *[({n: FAKE + 8}, INVALID) for n in ("q", "kc", "vc", "out")],
    *[({n: FAKE + 2}, INVALID) for n in ("table", "lens", "sel", "lse")],
    (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE), (dict(ws=FAKE + 16), INVALID),
    (dict(B=0, q=None, ws=None), OK),
])
def test_attention_rejects(lib, kw, rc):
    assert call(lib.mova_attention_paged, ATTEND, kw) == rc


def test_workspace_sizes(lib):
    sel, att = lib.mova_block_select_workspace_bytes, lib.mova_attention_workspace_bytes
    assert sel(4, 32, 8, 128, 100, 16, 8) >= 4 * 8 * 100 * 8 and sel(0, 32, 8, 128, 100, 16, 8) == 0
    for args in [(2049, 32, 8, 128, 100, 16, 8), (4, 33, 8, 128, 100, 16, 8), (4, 32, 8, 96, 100, 16, 8),
                 (4, 32, 8, 128, 0, 16, 8), (4, 32, 8, 128, 100, 0, 8), (-1, 32, 8, 128, 100, 16, 8),
                 (4, 32, 8, 128, 100, 16, -1), (4, 32, 8, 128, 1 << 28, 16, 8)]:
        assert sel(*args) == BAD and att(*args) == BAD, args
    assert sel(4, 32, 8, 128, 100, 16, 0) == BAD and att(4, 32, 8, 128, 100, 16, 0) != BAD
    assert att(4, 32, 8, 128, 100, 16, 0) % 256 == 0


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_checks(lib):
    """The binding refuses wrong types, shapes, strides and CPU tensors."""
    i32 = torch.int32
    q, pool, table, lens = z(2, 4, 64), z(5, 16, 2, 64), z(2, 3, dtype=i32), z(2, dtype=i32)
    att = binding.attention_paged
    for args, kw in [
        ((q.float(), pool, pool, table, lens, 1.0), {}),
        ((q, pool.float(), pool.float(), table, lens, 1.0), {}),
        ((q, pool, pool.to(torch.float8_e4m3fn), table, lens, 1.0), {}),
        ((q, pool, z(5, 16, 2, 128), table, lens, 1.0), {}),
        ((q.transpose(0, 1), pool, pool, table, lens, 1.0), {}),
        ((q, pool, pool, table.long(), lens, 1.0), {}),
        ((q, pool, pool, z(3, 3, dtype=i32), lens, 1.0), {}),
        ((q, pool, pool, table, lens, 1.0), dict(k_scale=z(3, dtype=torch.float32))),
        ((q, pool, pool, table, lens, 1.0), dict(sel_blocks=z(2, 3, 4, dtype=i32))),
        ((q, pool, pool, table, lens, 1.0), dict(sel_blocks=z(2, 2, 0, dtype=i32))),
        ((q, pool, pool, table, lens, 1.0), dict(lse=z(2, 2, dtype=torch.float32))),
        ((q, pool, pool, table, lens, 1.0), dict(out=z(2, 4, 128))),
        ((q, pool, pool, table, lens, 1.0), {}),  # on the CPU
    ]:
        with pytest.raises(ValueError):
            att(*args, **kw)
    with pytest.raises(binding.MovaError):
        att(z(2, 5, 64), pool, pool, table, lens, 1.0)
    kb = z(5, 2, 2, 64)
    for args in [(q, kb.float(), 16, table, lens, 2), (q, z(5, 2, 3, 64), 16, table, lens, 2),
                 (q, kb, 16, table, lens.long(), 2), (q, kb, 16, table, lens, 2)]:
        with pytest.raises(ValueError):
            binding.block_select(*args)
    with pytest.raises(binding.MovaError):
        binding.block_select(q, kb, 16, table, lens, 0)
    k, slots = z(3, 2, 64), z(3, dtype=torch.int64)
    for args, kw in [((k, None, None, pool, slots), {}), ((None, None, None, None, slots), {}),
                     ((k, k, pool, pool.to(torch.float8_e4m3fn), slots), {}),
                     ((k, z(4, 2, 64), pool, pool, slots), {}), ((k, k, pool, pool, slots.int()), {}),
                     ((k, k, pool, pool, slots), dict(k_bounds=z(5, 2, 64))),
                     ((k, k, pool, pool, slots), dict(v_scale=z(2))), ((k, k, pool, pool, slots), {})]:
        with pytest.raises(ValueError):
            binding.kv_store_paged(*args, **kw)
    free, count = z(9, dtype=i32), z(1, dtype=i32)
    for args, kw in [((lens, lens, -1, 16, table, free, count), {}),
                     ((lens.long(), lens, 2, 16, table, free, count), {}),
                     ((lens, lens, 2, 16, table, free, z(2, dtype=i32)), {}),
                     ((lens, lens, 2, 16, table, free, count), dict(slot_mapping=slots)),
                     ((lens, lens, 2, 16, table, free, count), {})]:
        with pytest.raises(ValueError):
            binding.paged_plan(*args, **kw)
