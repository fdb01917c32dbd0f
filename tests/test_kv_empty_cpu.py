"""Empty calls of the cache: nothing to do is GDN_OK, and launches nothing."""
import pytest

from speculative_verify_gdn_amd import gdn
from tests.test_kv_cpu import call, lib  # noqa: F401


@pytest.mark.parametrize("name,kw", [
    ("gdn_kv_fork", dict(B=0, n=0)), ("gdn_kv_fork", dict(B=0, n=0, src=None, table=None, pool=None)),
    ("gdn_kv_free", dict(B=0)), ("gdn_kv_free", dict(B=0, n=0)), ("gdn_kv_reserve", dict(B=0, lens=None)),
    ("gdn_kv_append", dict(B=0)), ("gdn_kv_rollback_tree", dict(B=0, node=None)), ("gdn_attn_verify", dict(B=0))])
def test_ok(lib, name, kw):  # noqa: F811
    assert call(lib, name, **kw) == gdn.GDN_OK


@pytest.mark.parametrize("kw", [dict(B=0, n=1), dict(B=-1, n=0), dict(B=0, n=0, P=0)])
def test_refused(lib, kw):  # noqa: F811
    assert call(lib, "gdn_kv_fork", **kw) == gdn.GDN_EINVAL


COPY = "gdn_kv_copy"


@pytest.mark.parametrize("kw", [
    dict(n=2 ** 31 - 1, planes=65535, Hkv=128, page=1024, D=256),           # 2^59 pieces of 16 KB and more
    dict(n=2 ** 26, planes=65535, Hkv=8, page=1024, D=256, dtype=gdn.GDN_F32)])
def test_copies_that_cannot_be_counted_are_refused(lib, kw):  # noqa: F811
    assert call(lib, COPY, **kw) == gdn.GDN_EUNSUPPORTED
    assert lib.gdn_last_error().decode().startswith(COPY)
