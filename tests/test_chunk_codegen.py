"""Checks on the gfx950 machine code of the chunk attention (CPU only: compiles
to assembly, runs nothing)."""
import re

import pytest

from test_paged_codegen import kernels


def joined(name, prefix):
    return {k: "\n".join(ins) for k, ins in kernels(name, prefix).items()}


@pytest.fixture(scope="module")
def many():
    return joined("chunk_attention.hip", "_ZN4mova22chunk_attention_kernel")


@pytest.fixture(scope="module")
def few():
    return joined("chunk_few.hip", "_ZN4mova16chunk_few_kernel")


def test_variants(many, few):
    """Of many rows: widths by types; of few: those by tracks."""
    assert len(many) == 6 and len(few) == 18


def test_products_and_transposed_reads(many, few):
    for name, text in many.items():
        assert "v_mfma_f32_32x32x16" in text and "ds_read_b64_tr_b16" in text, name
    for name, text in few.items():
        assert "v_mfma_f32_16x16x32" in text and "ds_read_b64_tr_b" in text, name


def test_8_bit_pools_are_multiplied_as_halves(many):
    for name, text in many.items():
        fp8 = "ELb1E" in name
        assert ("v_mfma_f32_32x32x16_f16" in text) == fp8, name


def test_few_rows_are_streamed_by_direct_loads(few):
    for name, text in few.items():
        assert "global_load_lds_dwordx4" in text, name
        assert re.search(r"s_waitcnt vmcnt\([1-9]\d*\)", text), f"{name}: the ring is drained"


def test_no_packed_fp32(many, few):
    for texts in (many, few):
        for name, text in texts.items():
            assert not re.search(r"\bv_pk_(?:add|mul|fma)_f32\b", text), name
