"""Pairs of neighbours where a workgroup takes many tokens, where the reads go past
the caches, and on the way into the cache."""
import random

import pytest
import torch

from speculative_verify_gdn_amd import gdn
from tests import window_ref as ref
from tests.test_gpu_rope import BF, F32, _gpu, check, dev, freqs_of, randn, say, trees  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode", ["pos", "lens", "tree"])
@pytest.mark.parametrize("B,K,H,D,rot", [(40, 600, 2, 64, 64), (301, 41, 3, 96, 24), (1, 9001, 1, 48, 22), (700, 13, 1, 512, 512),
                                         (5000, 3, 1, 16, 2), (90, 200, 2, 128, 32), (61, 301, 1, 80, 40), (2500, 5, 1, 64, 20)])
def test_many_tokens(B, K, H, D, rot, mode, dtype):
    say("neighbours, many tokens", B, K, H, D, rot, mode, dtype)
    if mode == "tree" and K > 64:
        B, K = B * K // 50 + 1, 50
    g, r = torch.Generator().manual_seed(B), random.Random(K)
    x, f = randn(g, B, K, H, D, dtype=dtype), freqs_of(rot)
    kw = dict(lens=[r.choice([0, -3, 77, 200000]) for _ in range(B)])
    if mode == "pos":
        kw["pos"] = [[r.randint(-5000, 100000) for _ in range(K)] for _ in range(B)]
    if mode == "tree":
        kw["parent"] = trees(B, K, D)
    count = [r.choice([0, 1, K, K + 7]) for _ in range(B)]
    y = torch.full((B, K, H, D), 9.0, dtype=dtype).cuda()
    gdn.rope(x.cuda(), y, f.cuda(), count=dev(count), interleaved=True, mscale=1.2, **{k: dev(v) for k, v in kw.items()})
    want, off = ref.turned(x, ref.positions(B, K, **kw), f, True, 1.2)
    there = torch.arange(K)[None] < torch.tensor(count)[:, None]
    got = y.cpu()
    check(got, want, off, dtype, there)
    assert torch.equal(got[..., rot:][there], x[..., rot:][there])
    assert bool((got[~there] == 9.0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved,norm", [(True, False), (True, True), (False, False)])
@pytest.mark.parametrize("H,D,rot", [(32, 128, 128), (16, 256, 64), (3, 128, 64)])
def test_large_windows(H, D, rot, norm, interleaved, dtype):
    """More than 48 MB of heads, many a token and few."""
    say("large windows", H, D, rot, norm, interleaved, dtype)
    B = 3
    K = 27_000_000 // (2 if dtype == F32 else 1) // (B * (H + norm) * D) + 1
    g = torch.Generator().manual_seed(D + H)
    x, f = randn(g, B, K, H, D, dtype=dtype), freqs_of(rot)
    lens, there = [0, 9, 100000], torch.ones(B, K, dtype=torch.bool)
    y = torch.empty(B, K, H, D, dtype=dtype, device="cuda")
    w = torch.randn(D, generator=g) if norm else None
    kw = dict(lens=dev(lens), interleaved=interleaved, mscale=0.8)
    if norm:
        k, ko = x[:, :, :1], torch.empty(B, K, 1, D, dtype=dtype, device="cuda")
        gdn.qk_norm_rope(x.cuda(), k.cuda(), w.cuda(), w.cuda(), f.cuda(), y, ko, **kw)
        assert torch.equal(ko, y[:, :, :1])
    else:
        gdn.rope(x.cuda(), y, f.cuda(), **kw)
    want, off = ref.turned(x, ref.positions(B, K, lens=lens), f, interleaved, 0.8, w)
    check(y.cpu(), want, off, dtype, there)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("B,K,Hq,Hkv,D,rot", [(1, 1, 16, 2, 256, 64), (3, 5, 4, 2, 64, 64), (2, 64, 6, 3, 128, 32), (9, 16, 2, 1, 64, 30),
                                              (2, 1700, 2, 1, 64, 20), (1, 3000, 1, 1, 64, 64)])
def test_append(B, K, Hq, Hkv, D, rot, norm, dtype):
    """Keys into the pages and queries beside them, with a factor on sine and cosine."""
    say("neighbours, append", B, K, Hq, Hkv, D, rot, norm, dtype)
    g = torch.Generator().manual_seed(K + D)
    page, lens = 16, [3 + 20 * b for b in range(B)]
    P = (lens[-1] + K) // page + 1
    table = torch.randperm(B * P, generator=g).view(B, P).tolist()
    q, k, v = (randn(g, B, K, h, D, dtype=dtype) for h in (Hq, Hkv, Hkv))
    wq, wk = (1 + 0.3 * torch.randn(D, generator=g) if norm else None for _ in range(2))
    parent = trees(B, K, K) if 1 < K <= 64 else None
    f = freqs_of(rot)
    pool = torch.full((2, B * P, Hkv, page, D), 7.0, dtype=dtype, device="cuda")
    qo = torch.empty(B, K, Hq, D, dtype=dtype, device="cuda")
    up = lambda t: None if t is None else t.cuda()
    gdn.kv_append_rope(k.cuda(), v.cuda(), pool[0], pool[1], dev(lens), dev(table), f.cuda(), q=q.cuda(), q_out=qo, wq=up(wq),
                       wk=up(wk), parent=None if parent is None else dev(parent), interleaved=True, mscale=1.3)
    at = torch.tensor(lens)[:, None] + torch.arange(K)                         # [B][K] slots
    page_of = torch.gather(torch.tensor(table), 1, at // page)
    keys, values = (plane.cpu()[page_of, :, at % page] for plane in pool)     # [B][K][Hkv][D]
    assert torch.equal(values, v)
    where, there = ref.positions(B, K, lens=lens, parent=parent), torch.ones(B, K, dtype=torch.bool)
    for got, x, w in ((qo.cpu(), q, wq), (keys, k, wk)):
        want, off = ref.turned(x, where, f, True, 1.3, w)
        check(got, want, off, dtype, there)
    used = torch.zeros(B * P, page, dtype=torch.bool)
    used[page_of, at % page] = True
    assert bool((pool.cpu().transpose(2, 3)[:, ~used] == 7.0).all())
