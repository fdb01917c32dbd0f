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
