"""Frequencies of the rotary pairs at the edges of their arguments."""
import math
import os

import pytest
import torch

from speculative_verify_gdn_amd import gdn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(gdn.LIB_PATH):
        pytest.skip("libgdn.so not built")
    gdn.load()


EDGES = [dict(scaling="yarn", factor=2.0, low=1e-310, high=32.0, original=4096.0),                          # high / low is no double
         dict(scaling="yarn", factor=2.0, low=1.9999999999999998, high=2.0, original=4 * math.pi),          # nor above 1 here
         dict(scaling="ntk", factor=1e200, rot=4), dict(scaling="ntk", factor=4.0, rot=4, base=1e308),
         dict(scaling="bands", factor=2.0, low=1e-310, high=32.0, original=4096.0),
         dict(scaling="linear", factor=1e300), dict(scaling="yarn", factor=1e300, original=1e300), dict(base=1e308),
         dict(scaling="ntk", factor=1e100, rot=512)]


@pytest.mark.parametrize("kw", EDGES)
def test_numbers_or_a_refusal(kw):
    """Every pair turns by a number above 0 (2^-1000 of a position is one too), or the call is refused."""
    try:
        f, m = gdn.rope_freqs(**dict(dict(rot=8, device="cpu"), **kw))
    except gdn.GdnError as e:
        assert e.code == gdn.GDN_EUNSUPPORTED and kw["scaling"] in ("ntk", "yarn")
        return
    assert math.isfinite(m) and bool(torch.isfinite(f).all()) and bool((f > 0).all()) and bool((f <= 1).all())


# (rot, base, original context, factor): of usual models, and ones whose bounds leave the pairs
SCALED = [(128, 1e6, 32768, 4.0), (64, 1e7, 262144, 4.0), (128, 1e4, 4096, 16.0), (64, 150000.0, 4096, 32.0), (64, 1e4, 4096, 40.0),
          (32, 5e5, 8192, 8.0), (16, 1e4, 100, 2.0), (64, 2.0, 4096, 8.0), (512, 1e4, 2048, 8.0), (2, 1e4, 4096, 2.0),
          (4, 1e4, 1e12, 2.0)]


@pytest.mark.parametrize("low,high", [(1.0, 32.0), (2.0, 3.0)])
@pytest.mark.parametrize("rot,base,original,factor", SCALED)
def test_yarn_between_rounded_bounds(rot, base, original, factor, low, high):
    """The ramp over the pairs' indices from the last whole pair of `high` turns to the first one of `low`."""
    f, m = gdn.rope_freqs(rot, base, "yarn_rounded", factor, low=low, high=high, original=original, device="cpu")
    i = torch.arange(rot // 2, dtype=torch.float64)
    plain = torch.tensor([base ** (-2.0 * j / rot) for j in range(rot // 2)], dtype=torch.float64)
    turns = original * plain / (2 * math.pi)
    # the pair of n turns, from base^(-2 i / rot) original / 2 pi = n
    pair = lambda n: rot / 2 * math.log(original / (2 * math.pi * n), base)
    p, q = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
    part = ((i - p) / (q - p)).clamp(0, 1) if q > p else (i > p).double()     # of the division by the factor
    torch.testing.assert_close(f, plain * (1 - part) + plain * part / factor, rtol=1e-12, atol=0)
    assert m == pytest.approx(0.1 * math.log(factor) + 1, rel=2 ** -24)
    # whole pairs outside the turns' bounds are as without a ramp
    if pair(low) <= rot - 1 and pair(high) >= 0:
        torch.testing.assert_close(f[i <= p], plain[i <= p], rtol=1e-13, atol=0)
        torch.testing.assert_close(f[(i >= q) & (i > p)], plain[(i >= q) & (i > p)] / factor, rtol=1e-13, atol=0)
    # and the unrounded form meets it where the bounds are whole pairs
    lo, hi = (original / (2 * math.pi) * base ** (-2.0 * j / rot) for j in (min(q, rot // 2 - 1), p))
    if 0 <= p < q <= rot // 2 - 1:
        whole, _ = gdn.rope_freqs(rot, base, "yarn", factor, low=lo, high=hi, original=original, device="cpu")
        torch.testing.assert_close(f, whole, rtol=1e-12, atol=0)


def test_the_paper_s_ramp_is_bands():
    """Linear in the turns between 1 and 32 of them, as the paper has it."""
    rot, base, original, factor = 128, 1e4, 4096, 16.0
    f, m = gdn.rope_freqs(rot, base, "bands", factor, low=1.0, high=32.0, original=original, device="cpu")
    plain = torch.tensor([base ** (-2.0 * j / rot) for j in range(rot // 2)], dtype=torch.float64)
    ramp = ((original * plain / (2 * math.pi) - 1) / 31).clamp(0, 1)
    torch.testing.assert_close(f, (1 - ramp) * plain / factor + ramp * plain, rtol=1e-12, atol=0)
    assert m == 1.0


@pytest.mark.parametrize("kw", [dict(original=0.0), dict(original=4096.0, low=4.0, high=4.0), dict(original=4096.0, low=0.0),
                                dict(original=4096.0, factor=0.5)])
def test_yarn_rounded_refused(kw):
    with pytest.raises(gdn.GdnError) as e:
        gdn.rope_freqs(64, scaling="yarn_rounded", device="cpu", **kw)
    assert e.value.code == gdn.GDN_EINVAL


def test_no_scaling_behind_the_last():
    import ctypes

    f, m = (ctypes.c_double * 4)(), ctypes.c_float()
    args = lambda code: (8, 1e4, code, 2.0, 1.0, 32.0, 4096.0, f, ctypes.byref(m))
    assert gdn.load().gdn_rope_freqs(*args(5)) == gdn.GDN_OK
    assert gdn.load().gdn_rope_freqs(*args(6)) == gdn.GDN_EINVAL
    assert gdn.load().gdn_rope_freqs(*args(-1)) == gdn.GDN_EINVAL
