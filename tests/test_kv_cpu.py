"""Refusals of the paged cache calls and the window attention: every bad
argument is turned down on the host, with its code, before anything is
launched, by the C ABI (fake addresses) and by the binding (CPU tensors)."""
import ctypes
import os

import pytest
import torch

from speculative_verify_gdn_amd import gdn

A, MB = 0x7F0000000000, 1 << 24
E, U = gdn.GDN_EINVAL, gdn.GDN_EUNSUPPORTED
BF, F32 = gdn.GDN_BF16, gdn.GDN_F32


def p(i, off=0):
    return ctypes.c_void_p(A + i * 64 * MB + off)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        pytest.skip("libgdn.so not built")
    return gdn.load()


GEOM = dict(Hkv=2, page=16, D=64, dtype=BF)
CALLS = {
    "gdn_kv_reserve": ("lens add table ref granted B P n_pages page",
                       dict(lens=p(1), add=p(2), table=p(3), ref=p(4), granted=p(5), B=2, P=4, n_pages=8, page=16)),
    "gdn_kv_append": ("k v kv_stride k_pages v_pages lens count table B K Hkv D page n_pages P dtype",
                      dict(GEOM, k=p(1), v=p(2), kv_stride=128, k_pages=p(3), v_pages=p(4), lens=p(5), count=p(6),
                           table=p(7), B=2, K=3, n_pages=8, P=4)),
    "gdn_kv_rollback_tree": ("node parent lens count table ref pool lens_out B N P planes n_pages Hkv page D dtype",
                             dict(GEOM, node=p(1), parent=p(2), lens=p(3), count=p(4), table=p(5), ref=p(6), pool=p(7),
                                  lens_out=p(8), B=2, N=4, P=4, planes=2, n_pages=8)),
    "gdn_kv_free": ("rows lens table ref n B P n_pages",
                    dict(rows=p(1), lens=p(2), table=p(3), ref=p(4), n=1, B=2, P=4, n_pages=8)),
    "gdn_kv_fork": ("src dst lens table ref pool granted n B P planes n_pages Hkv page D dtype",
                    dict(GEOM, src=p(1), dst=p(2), lens=p(3), table=p(4), ref=p(5), pool=p(6), granted=p(7), n=1, B=2,
                         P=4, planes=2, n_pages=8)),
    "gdn_kv_compact": ("table ref pool table_out ref_out workspace workspace_bytes entries planes n_pages Hkv page D dtype",
                       dict(GEOM, table=p(1), ref=p(2), pool=p(3), table_out=p(4), ref_out=p(5), workspace=p(6),
                            workspace_bytes=1 << 20, entries=8, planes=2, n_pages=8)),
    "gdn_kv_copy": ("src dst pool n planes n_pages Hkv page D dtype",
                    dict(GEOM, src=p(1), dst=p(2), pool=p(3), n=1, planes=2, n_pages=8)),
    "gdn_attn_verify": ("q q_stride k_pages v_pages lens count parent table o lse workspace workspace_bytes B K Hq Hkv "
                        "D page n_pages P prefix_len scale dtype",
                        dict(GEOM, q=p(1), q_stride=256, k_pages=p(2), v_pages=p(3), lens=p(4), count=p(5), parent=p(6),
                             table=p(7), o=p(8), lse=p(9), workspace=p(10), workspace_bytes=1 << 30, B=2, K=3, Hq=4,
                             n_pages=8, P=4, prefix_len=0, scale=0.125)),
}


def call(lib, name, **kw):
    order, args = CALLS[name]
    args = dict(args, **kw)
    return getattr(lib, name)(*[args[a] for a in order.split()], None)


BAD_GEOM = [(dict(D=96), U), (dict(page=24), U), (dict(page=8), U), (dict(page=2048), U), (dict(page=0), E),
            (dict(dtype=3), E), (dict(Hkv=0), E), (dict(n_pages=0), E), (dict(n_pages=1 << 22), U)]
BAD = {
    "gdn_kv_reserve": [(dict(lens=None), E), (dict(ref=None), E), (dict(table=p(3, 2)), E), (dict(B=-1), E),
                       (dict(P=0), E), (dict(B=70000), U), (dict(page=48), U), (dict(n_pages=0), E),
                       (dict(granted=p(1)), E), (dict(ref=p(3, 8)), E)],
    "gdn_kv_append": BAD_GEOM + [(dict(k=None), E), (dict(table=None), E), (dict(k=p(1, 8)), E), (dict(lens=p(5, 2)), E),
                                 (dict(kv_stride=120), E), (dict(kv_stride=132), E), (dict(K=0), E), (dict(B=-1), E),
                                 (dict(v_pages=p(3)), E), (dict(k=p(3)), E), (dict(k_pages=p(7)), E)],
    "gdn_kv_rollback_tree": BAD_GEOM + [(dict(node=None), E), (dict(pool=None), E), (dict(pool=p(7, 4)), E),
                                        (dict(N=0), E), (dict(N=65), U), (dict(planes=0), E), (dict(lens_out=p(1)), E),
                                        (dict(lens_out=p(3, 4)), E), (dict(ref=p(5, 16)), E), (dict(table=p(3)), E)],
    "gdn_kv_free": [(dict(rows=None), E), (dict(ref=None), E), (dict(rows=p(1, 1)), E), (dict(n=-1), E), (dict(P=0), E),
                    (dict(lens=p(1)), E), (dict(n_pages=0), E)],
    "gdn_kv_fork": BAD_GEOM + [(dict(src=None), E), (dict(granted=None), E), (dict(n=-1), E), (dict(n=5000), U),
                               (dict(B=0), E), (dict(granted=p(1)), E), (dict(lens=p(2)), E), (dict(pool=p(6, 2)), E)],
    "gdn_kv_compact": BAD_GEOM + [(dict(ref=None), E), (dict(workspace=None), E), (dict(workspace_bytes=16), E),
                                  (dict(table_out=p(1)), E), (dict(ref_out=p(2)), E), (dict(entries=-1), E),
                                  (dict(workspace=p(6, 8)), E), (dict(table=None), E)],
    "gdn_kv_copy": BAD_GEOM + [(dict(src=None), E), (dict(pool=None), E), (dict(n=-1), E), (dict(src=p(3)), E),
                               (dict(dst=p(2, 2)), E)],
    "gdn_attn_verify": BAD_GEOM + [(dict(q=None), E), (dict(o=None), E), (dict(workspace=None), E), (dict(table=None), E),
                                   (dict(q=p(1, 8)), E), (dict(lse=p(9, 2)), E), (dict(q_stride=255), E),
                                   (dict(q_stride=260), E), (dict(K=0), E), (dict(K=65), U), (dict(Hq=3), E),
                                   (dict(B=5000), U), (dict(prefix_len=8), E), (dict(prefix_len=-16), E),
                                   (dict(prefix_len=80), E), (dict(scale=float("nan")), E), (dict(workspace_bytes=8), E),
                                   (dict(scale=float("inf")), E), (dict(o=p(1)), E), (dict(lse=p(8)), E),
                                   (dict(o=p(3)), E), (dict(workspace=p(7)), E), (dict(P=1 << 28), U)],
}


@pytest.mark.parametrize("name,kw,code", [(n, kw, c) for n in BAD for kw, c in BAD[n]])
def test_refused_on_the_host(lib, name, kw, code):
    assert call(lib, name, **kw) == code
    assert lib.gdn_last_error().decode().startswith(name)


@pytest.mark.parametrize("name,kw", [("gdn_kv_reserve", dict(B=0)), ("gdn_kv_append", dict(B=0, k=None)),
                                     ("gdn_kv_rollback_tree", dict(B=0)), ("gdn_kv_free", dict(n=0)),
                                     ("gdn_kv_fork", dict(n=0)), ("gdn_kv_copy", dict(n=0)),
                                     ("gdn_attn_verify", dict(B=0, q=None))])
def test_empty_calls_are_ok(lib, name, kw):
    assert call(lib, name, **kw) == gdn.GDN_OK


def test_workspace_sizes(lib):
    n = ctypes.c_size_t(0)
    assert lib.gdn_kv_compact_workspace(100, ctypes.byref(n)) == gdn.GDN_OK and n.value >= 8 * 100
    assert lib.gdn_kv_compact_workspace(0, ctypes.byref(n)) == E
    assert lib.gdn_kv_compact_workspace(8, None) == E
    sizes = [4, 8, 16, 4, 128, 16, 64, 0, BF]
    assert lib.gdn_attn_workspace(*sizes, ctypes.byref(n)) == gdn.GDN_OK and n.value > 0
    assert lib.gdn_attn_workspace(*sizes[:-1], 9, ctypes.byref(n)) == E
    assert lib.gdn_attn_workspace(*sizes, None) == E


def test_binding_refuses_before_the_library():
    i = torch.zeros(2, dtype=torch.int32)
    table = torch.full((2, 4), -1, dtype=torch.int32)
    pool = torch.zeros(2, 8, 2, 16, 64, dtype=torch.bfloat16)
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):   # CPU tensors
        gdn.kv_reserve(i, i, table, i, 16, i)
    with pytest.raises(ValueError):
        gdn.kv_copy(i, i, pool)
    with pytest.raises(ValueError):
        gdn.attn_verify(q, pool[0], pool[1], i, table, q.clone(), workspace=torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        gdn.kv_rollback_tree(i, None, i, table, i, pool, i, N=4)
