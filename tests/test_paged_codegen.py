"""Checks on the gfx950 machine code of the paged cache's kernels (CPU only).

* Attention and block scores keep several tiles in flight: the waits before
  their LDS reads leave whole groups of direct loads outstanding, and no wait
  for all of them stands between the products of a tile.
* Both contract on the matrix units, attention's values through transposing
  LDS reads, and read the cache with the non-temporal hint where a row fills a
  cache line and no two waves read it.
"""
import os
import re

import pytest

from mixture_value_projection_amd import build


def kernels(name, prefix):
    text = build.device_asm(os.path.join(build.CSRC, name))
    out = {}
    for m in re.finditer(rf"^({prefix}\w*):", text, re.M):
        body = text[m.start():text.find(".end_amdhsa_kernel", m.start())]
        out[m.group(1)] = [l.strip() for l in body.splitlines()
                           if l.strip() and not l.strip().startswith((";", "."))]
    assert out, prefix
    return out


@pytest.fixture(scope="module")
def attention():
    return kernels("attention.hip", "_ZN4mova16attention_kernel")


@pytest.fixture(scope="module")
def scores():
    return kernels("block_select.hip", "_ZN4mova19select_score_kernel")


def test_rings_stay_in_flight(attention, scores):
    for name, ins in {**attention, **scores}.items():
        assert any(re.match(r"s_waitcnt vmcnt\([1-9]\d*\)", i) for i in ins), name
        products = [n for n, i in enumerate(ins) if i.startswith("v_mfma")]
        # From a tile's first product to the next refill of the ring.
        tile = ins[products[0]:products[-1]]
        drained = [i for i in tile if re.match(r"s_waitcnt.*vmcnt\(0\)", i)]
        loads = [i for i in tile if i.startswith("global_load_dword")]
        if not loads:  # (queries of groups above 16 are read inside the scores' tile)
            assert not drained, f"{name}: {drained}"


def test_attention_reads_values_transposed(attention):
    assert len(attention) == 60  # head_dim x dtype x (tracks of a workgroup, shared) x list
    for name, ins in attention.items():
        D, fp8, shared = (int(x) for x in
                          re.search(r"ILi(\d+)ELb([01])ELi\dELb([01])E", name).groups())
        assert any(i.startswith("ds_read_b64_tr_b8" if fp8 else "ds_read_b64_tr_b16") for i in ins)
        assert any(i.startswith("v_mfma_f32_16x16x32_bf16") for i in ins), name
        hinted = [bool(re.search(r" nt\b", i)) for i in ins if i.startswith("global_load_lds_dwordx4")]
        assert hinted and set(hinted) == {not shared and not (fp8 and D == 64)}, name


def test_no_packed_fp32(attention, scores):
    for name, ins in {**attention, **scores}.items():
        assert not any(re.match(r"v_pk_(add|mul|fma)_f32", i) for i in ins), name
