"""Decode attention over infinite, NaN and very large values that take part,
against the 64-bit softmax and with the tolerances of tests/pagedlib.py.  Sums
above 2^112 are formed with weights to 2^-15 instead of the 2^-16 counted there;
the 2^-16 more is part of the 2^-13 that is counted for chains of 2^11 terms,
of which these shapes have at most 2^10 (2^-14)."""
import math

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


# lens, Hq, H, D, bs: single keys, rows of one workgroup, rows split among many,
# one and several tracks of a key head, every tile shape.
SHAPES = [
    ([1], 4, 1, 128, 16),
    ([1, 2, 17, 0, 33], 8, 2, 64, 16),
    ([1, 40, 130], 8, 2, 256, 16),
    ([130, 1], 32, 8, 128, 16),
    ([3000, 700], 32, 8, 128, 16),
    ([9000], 4, 2, 64, 32),
    ([5000], 4, 1, 256, 32),
    ([900, 333], 32, 1, 64, 16),
    ([2500, 60], 40, 1, 128, 64),
    ([700, 12], 6, 3, 128, 24),
]
# Largest v of the softmax's sum; bf16's largest finite value is 3.39e38.
LARGE = 3e38


def check(a, what, window=0, sel=None):
    out, lse = C.run_attention(a, window, sel)
    want, wlse, tol, tlse = R.attention(a["q"], a["k"], a["v"], a["table"], a["lens"],
                                        a["q"].shape[2] ** -0.5, None, None, window, sel)
    out = out.double()
    fine = want.isfinite()
    assert torch.equal(out.isnan(), want.isnan()), f"{what}: NaN"
    infinite = want.isinf()
    assert torch.equal(out[infinite], want[infinite]), f"{what}: infinities"
    assert ((out - want).abs()[fine] <= tol[fine]).all(), \
        f"{what}: off by {float(((out - want).abs() - tol)[fine].max()):.3g} too much"
    full = wlse != -math.inf
    assert ((lse.double() - wlse).abs()[full] <= tlse[full]).all(), f"{what}: lse"
    assert (lse[~full] == -math.inf).all(), f"{what}: lse of empty rows"


def lists(a, H, n):
    rng = np.random.default_rng(n)
    return rng.integers(-1, a["table"].shape[1], (len(a["lens"]), H, n))


def each_form(a, H, what):
    check(a, what)
    check(a, what + ", window", window=50)
    check(a, what + ", listed", sel=lists(a, H, 9))


def slots_of(a, b):
    bs = a["k"].shape[1]
    p = np.arange(a["lens"][b])
    return a["table"][b, p // bs], p % bs


@pytest.mark.parametrize("lens,Hq,H,D,bs", SHAPES)
def test_infinite_values(lens, Hq, H, D, bs):
    """An infinite value of a key with any weight makes its channel infinite,
    two of unlike signs or a NaN make it NaN; the other channels stay as they
    are."""
    a = C.make_attention(11 + D, lens, Hq, H, D, bs, torch.bfloat16)
    rng = np.random.default_rng(D)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        page, row = slots_of(a, b)
        at = rng.integers(0, n, 6)
        a["v"][page[at[0]], row[at[0]], :, 3] = math.inf
        a["v"][page[at[1]], row[at[1]], :, 5] = -math.inf
        a["v"][page[at[2]], row[at[2]], :, D - 1] = math.inf
        a["v"][page[at[3]], row[at[3]], :, 20] = math.nan
        a["v"][page[at[4]], row[at[4]], :, 30] = math.inf
        a["v"][page[at[5]], row[at[5]], :, 30] = -math.inf
    each_form(a, H, "infinities")
    # Nothing but infinities in a channel.
    a["v"][:, :, :, 8] = math.inf
    a["v"][:, :, :, 9] = -math.inf
    each_form(a, H, "channels of infinities")


@pytest.mark.parametrize("lens,Hq,H,D,bs", SHAPES)
def test_large_values(lens, Hq, H, D, bs):
    """Values whose sum over the keys passes the largest fp32 number, while
    their weighted mean does not."""
    a = C.make_attention(12 + D, lens, Hq, H, D, bs, torch.bfloat16)
    a["v"][:] = LARGE
    each_form(a, H, "equal")
    rng = np.random.default_rng(D)
    a["v"] = torch.from_numpy(rng.uniform(-LARGE, LARGE, a["v"].shape)).to(torch.bfloat16)
    each_form(a, H, "either sign")
    # A few large ones, in the last rows of a request only, and one infinity.
    a = C.make_attention(13 + D, lens, Hq, H, D, bs, torch.bfloat16)
    for b, n in enumerate(lens):
        page, row = slots_of(a, b)
        for i in range(max(0, n - 3), n):
            a["v"][page[i], row[i], :, ::3] = LARGE
        if n:
            a["v"][page[n // 2], row[n // 2], :, 1] = -math.inf
    each_form(a, H, "few")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_just_below_the_second_pass(D):
    """Values of 2^112 and around: sums below and above where they are formed
    again, in different parts of one row."""
    a = C.make_attention(D, [4000, 3], 4, 2, D, 16, torch.bfloat16)
    rng = np.random.default_rng(D)
    size = torch.from_numpy(2.0 ** rng.integers(100, 122, a["v"].shape[0]))[:, None, None, None]
    a["v"] = (a["v"].double() * size).to(torch.bfloat16)
    each_form(a, 2, "between")


@pytest.mark.parametrize("dtype", [torch.bfloat16, C.FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("lens,Hq,H,D,bs", SHAPES)
def test_every_logit_minus_infinity(lens, Hq, H, D, bs, dtype):
    """Rows whose every logit is -infinity give zeros, whatever their values."""
    for v in (1.0, math.inf, math.nan):  # (the 8-bit type has NaN for infinity)
        a = C.make_attention(14, lens, Hq, H, D, bs, dtype)
        a["q"][:, :, 0] = -math.inf
        a["k"][:, :, :, 0] = torch.ones(1).to(dtype)
        a["v"][:] = torch.tensor(v).to(dtype)
        out, lse = C.run_attention(a)
        assert (out == 0).all() and (lse == -math.inf).all(), v
