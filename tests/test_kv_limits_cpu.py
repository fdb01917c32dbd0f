"""Sizes past what the kernels count in 32 bits are refused on the host."""
import ctypes

import pytest

from speculative_verify_gdn_amd import gdn
from tests.test_kv_cpu import BF, F32, U, call, lib, p  # noqa: F401


@pytest.mark.parametrize("name,kw", [
    ("gdn_kv_append", dict(K=65536, Hkv=1024, D=256, dtype=F32, kv_stride=1024 * 256)),
    ("gdn_kv_rollback_tree", dict(planes=65535, Hkv=1024, D=256, dtype=F32)),
    ("gdn_kv_fork", dict(planes=65535, Hkv=1024, D=256, dtype=F32)),
    ("gdn_kv_copy", dict(planes=65535, Hkv=1024, D=256, dtype=F32)),
    ("gdn_kv_free", dict(n=(1 << 20) + 1)),
    ("gdn_attn_verify", dict(B=4096, K=64, Hq=1024, Hkv=1, D=256, q_stride=1024 * 256)),
])
def test_refused(lib, name, kw):  # noqa: F811
    assert call(lib, name, **kw) == U
    assert lib.gdn_last_error().decode().startswith(name)


def test_workspace_refuses_what_the_call_would(lib):  # noqa: F811
    n = ctypes.c_size_t(0)
    assert lib.gdn_attn_workspace(4096, 64, 1024, 1, 256, 16, 4, 0, BF, ctypes.byref(n)) == gdn.GDN_EUNSUPPORTED
    assert lib.gdn_attn_workspace(256, 64, 1024, 1, 256, 16, 4, 0, BF, ctypes.byref(n)) == gdn.GDN_OK
