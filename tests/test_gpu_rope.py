"""The rotary calls on the GPU against the 64-bit plain forms of window_ref.py:
layouts, parts of a head, positions, strides, trees, ragged windows, the cache."""
import math
import random

import pytest
import torch

from speculative_verify_gdn_amd import gdn
from tests import kv_ref, window_ref as ref

pytestmark = pytest.mark.gpu
I32, BF, F32 = torch.int32, torch.bfloat16, torch.float32


def say(*a):
    print("[gpu case]", *a, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.load()
    yield
    torch.cuda.synchronize()


def dev(x):
    return torch.tensor(x, dtype=I32).cuda()


def trees(B, K, seed, forest=True):
    r = random.Random(seed)
    return [[r.randint(-2 if forest else 0, t - 1) if t else -1 for t in range(K)] for b in range(B)]


def randn(g, *shape, dtype):
    return (torch.randn(*shape, generator=g) * 1.5).to(dtype)


def freqs_of(rot, base=10000.0):
    return torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)


def check(got, want, off, dtype, there):
    """Within the bound where `there` [B][K], NaN nowhere."""
    bound = ref.rounded(off, want, dtype)
    d = ((got.double() - want).abs() / bound)[there]
    assert not bool(d.isnan().any())
    assert d.numel() == 0 or float(d.max()) <= 1.0, float(d.max())


# heads of every kind: whole, part, pairs that fill no 16 bytes, the largest
HEADS = [(64, 64), (128, 32), (256, 64), (256, 256), (80, 80), (96, 24), (192, 192), (16, 2), (16, 16), (512, 512), (112, 38),
         (512, 6), (48, 46), (512, 20), (80, 40), (256, 12)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", HEADS)
def test_rope_heads(D, rot, interleaved, dtype):
    say("rope", D, rot, interleaved, dtype)
    g = torch.Generator().manual_seed(D + rot)
    B, K, H = 2, 5, 3
    x, f = randn(g, B, K, H, D, dtype=dtype), freqs_of(rot)
    lens, count = [7, 1000], [5, 3]
    y = torch.full((B, K, H, D), 9.0, dtype=dtype).cuda()
    gdn.rope(x.cuda(), y, f.cuda(), lens=dev(lens), count=dev(count), interleaved=interleaved, mscale=1.25)
    want, off = ref.turned(x, ref.positions(B, K, lens=lens), f, interleaved, 1.25)
    there = torch.arange(K)[None] < torch.tensor(count)[:, None]
    got = y.cpu()
    check(got, want, off, dtype, there)
    assert torch.equal(got[..., rot:][there], x[..., rot:][there])   # the rest of the head: the same bits
    assert bool((got[~there] == 9.0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,K,H,mode", [(1, 1, 1, "none"), (1, 1, 40, "lens"), (3, 64, 2, "tree"), (5, 17, 7, "tree"), (2, 1000, 3, "lens"),
                                        (300, 1, 5, "pos"), (7, 33, 1, "pos"), (1, 5000, 2, "none"), (65, 64, 1, "tree"),
                                        (2500, 2, 1, "lens"), (1, 1, 1024, "pos")])
def test_rope_positions(B, K, H, mode, dtype):
    say("rope positions", B, K, H, mode, dtype)
    g = torch.Generator().manual_seed(B + K)
    r = random.Random(K)
    D, rot = 64, 32
    x, f = randn(g, B, K, H, D, dtype=dtype), freqs_of(rot, 500.0)
    lens = None if mode == "none" else [r.choice([0, -3, 12, 4095]) for _ in range(B)]
    parent = trees(B, K, B) if mode == "tree" else None
    pos = [[r.randint(-5000, 5000) for _ in range(K)] for _ in range(B)] if mode == "pos" else None
    count = [r.randint(-1, K + 1) for _ in range(B)] if K > 1 else None
    y = torch.full((B, K, H, D), 9.0, dtype=dtype).cuda()
    opt = lambda v: None if v is None else dev(v)
    gdn.rope(x.cuda(), y, f.cuda(), pos=opt(pos), lens=opt(lens), parent=opt(parent), count=opt(count))
    want, off = ref.turned(x, ref.positions(B, K, pos, lens, parent), f)
    there = torch.arange(K)[None] < torch.tensor(count or [K] * B)[:, None]
    check(y.cpu(), want, off, dtype, there)
    assert bool((y.cpu()[~there] == 9.0).all())


def test_far_positions():
    """Positions to the ends of 32 bits: the angle is formed in 64."""
    say("far positions")
    g = torch.Generator().manual_seed(3)
    pos = [[0, 1, -1, 2 ** 20 + 1, 10 ** 9 + 7, 2 ** 31 - 1, -2 ** 31]]
    x, f = randn(g, 1, 7, 4, 128, dtype=F32), freqs_of(128, 1e6)
    y = torch.empty_like(x, device="cuda")
    gdn.rope(x.cuda(), y, f.cuda(), pos=dev(pos))
    want, off = ref.turned(x, pos, f)
    check(y.cpu(), want, off, F32, torch.ones(1, 7, dtype=torch.bool))
    lens = [2 ** 31 - 1]                                     # a depth past the last length of 32 bits
    gdn.rope(x.cuda(), y, f.cuda(), lens=dev(lens))
    want, off = ref.turned(x, ref.positions(1, 7, lens=lens), f)
    check(y.cpu(), want, off, F32, torch.ones(1, 7, dtype=torch.bool))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,rot", [(128, 128), (48, 46)])
def test_rope_there_and_back(D, rot, dtype):
    """Turned by p and by -p in place: within two roundings of the start (the transpose of a turn is the turn back)."""
    say("rope back", D, rot, dtype)
    g = torch.Generator().manual_seed(1)
    x, f = randn(g, 3, 20, 4, D, dtype=dtype), freqs_of(rot)
    pos = torch.randint(0, 100000, (3, 20), generator=g).to(I32)
    y = x.cuda()
    gdn.rope(y, y, f.cuda(), pos=pos.cuda())
    once, off1 = ref.turned(x, pos.tolist(), f)
    check(y.cpu(), once, off1, dtype, torch.ones(3, 20, dtype=torch.bool))
    mid = y.cpu()
    gdn.rope(y, y, f.cuda(), pos=(-pos).cuda())
    back, off2 = ref.turned(mid, (-pos).tolist(), f)
    check(y.cpu(), back, off2, dtype, torch.ones(3, 20, dtype=torch.bool))
    # the way there rounded each element by half a step, which the way back adds up over a pair
    half = torch.finfo(dtype).eps / 2
    r = x.double().abs().amax(-1, keepdim=True)
    assert float(((y.cpu().double() - x.double()).abs() / r).max()) <= 6 * half + 64 * 2.0 ** -24


STRIDES = {
    "dense": lambda g, B, K, H, D, t: randn(g, B, K, H, D, dtype=t).cuda(),
    "slice": lambda g, B, K, H, D, t: randn(g, B, K, H * D + 3 * 32, dtype=t).cuda()[..., 32:32 + H * D].unflatten(-1, (H, D)),
    "heads first": lambda g, B, K, H, D, t: randn(g, B, H, K, D, dtype=t).cuda().transpose(1, 2),
    "tokens first": lambda g, B, K, H, D, t: randn(g, K, B, H, D, dtype=t).cuda().transpose(0, 1),
    "gated": lambda g, B, K, H, D, t: randn(g, B, K, H, 2, D, dtype=t).cuda()[:, :, :, 0],
    "repeated": lambda g, B, K, H, D, t: randn(g, B, K, 1, D, dtype=t).cuda().expand(B, K, H, D),
}


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("order", STRIDES)
def test_rope_strides(order, dtype):
    say("rope strides", order, dtype)
    g = torch.Generator().manual_seed(5)
    B, K, H, D = 3, 6, 4, 96
    x, f = STRIDES[order](g, B, K, H, D, dtype), freqs_of(32)
    want, off = ref.turned(x.cpu(), ref.positions(B, K), f)
    there = torch.ones(B, K, dtype=torch.bool)
    y = torch.empty(B, K, H, D, dtype=dtype, device="cuda")
    gdn.rope(x, y, f.cuda())
    check(y.cpu(), want, off, dtype, there)
    if order == "repeated":
        with pytest.raises(gdn.GdnError):                   # rows that meet cannot be written
            gdn.rope(y, x, f.cuda())
        return
    whole = x._base if x._base is not None else x
    before = whole.clone()
    touched = torch.zeros_like(whole, dtype=torch.bool)
    torch.as_strided(touched, x.shape, x.stride(), x.storage_offset()).fill_(True)
    gdn.rope(x, x, f.cuda())                                # in place, the elements between stay
    assert torch.equal(x, y)
    assert torch.equal(whole[~touched], before[~touched])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,K,Hq,Hk,D,rot", [(1, 1, 16, 2, 256, 64), (3, 8, 24, 4, 256, 256), (2, 5, 3, 3, 80, 40), (1, 3, 1, 1, 16, 0),
                                             (40, 16, 8, 1, 64, 64), (2, 700, 5, 2, 128, 96), (2, 3, 6, 2, 512, 512), (1, 2, 4, 2, 112, 38)])
def test_norm(B, K, Hq, Hk, D, rot, interleaved, dtype):
    say("norm", B, K, Hq, Hk, D, rot, interleaved, dtype)
    g = torch.Generator().manual_seed(D + K)
    row = randn(g, B, K, (Hq + 2 * Hk) * D, dtype=dtype)
    row[:, 0, :D] = 0                                        # a head of zeros
    row[-1, -1, D * Hq:D * Hq + D] *= 1e-3                   # a small one, where eps counts
    q, k = row[..., :Hq * D].unflatten(-1, (Hq, D)), row[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
    wq, wk = torch.randn(D, generator=g), 1 + 0.3 * torch.randn(D, generator=g)
    f = freqs_of(rot) if rot else torch.zeros(0, dtype=torch.float64)
    parent = trees(B, K, 1) if 1 < K <= 64 else None
    lens = [100 * b for b in range(B)]
    dr = row.cuda()
    dq, dk = dr[..., :Hq * D].unflatten(-1, (Hq, D)), dr[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
    qo, ko = (torch.empty(B, K, h, D, dtype=dtype, device="cuda") for h in (Hq, Hk))
    kw = dict(lens=dev(lens), parent=None if parent is None else dev(parent), eps=1e-5, interleaved=interleaved, mscale=0.75)
    gdn.qk_norm_rope(dq, dk, wq.cuda(), wk.cuda(), f.cuda() if rot else None, qo, ko, **kw)
    where = ref.positions(B, K, lens=lens, parent=parent)
    there = torch.ones(B, K, dtype=torch.bool)
    for got, x, w in ((qo, q, wq), (ko, k, wk)):
        want, off = ref.turned(x, where, f, interleaved, 0.75, w, 1e-5)
        check(got.cpu(), want, off, dtype, there)
    # dense q and k may be their own outputs
    cq, ck = dq.contiguous(), dk.contiguous()
    gdn.qk_norm_rope(cq, ck, wq.cuda(), wk.cuda(), f.cuda() if rot else None, cq, ck, **kw)
    assert torch.equal(cq, qo) and torch.equal(ck, ko)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_values_that_are_not_finite(interleaved, dtype):
    """NaN and infinities stay in their pair (without a norm) or their head (with one)."""
    say("not finite", interleaved, dtype)
    g = torch.Generator().manual_seed(2)
    D, rot = 64, 32
    x = randn(g, 1, 4, 3, D, dtype=dtype)
    clean, f = x.clone(), freqs_of(rot)
    x[0, 1, 1, 5], x[0, 2, 0, 40], x[0, 3, 2, 63] = math.nan, math.inf, -math.inf
    y, z = (torch.empty(1, 4, 3, D, dtype=dtype, device="cuda") for _ in range(2))
    gdn.rope(x.cuda(), y, f.cuda(), interleaved=interleaved)
    gdn.rope(clean.cuda(), z, f.cuda(), interleaved=interleaved)
    y, z = y.cpu(), z.cpu()
    same = (y == z)
    other = 4 if interleaved else 5 + rot // 2
    bad = torch.zeros_like(same)
    bad[0, 1, 1, 5] = bad[0, 1, 1, other] = bad[0, 2, 0, 40] = bad[0, 3, 2, 63] = True
    assert bool((same | bad).all())
    assert bool(y[0, 1, 1, 5].isnan()) and bool(y[0, 1, 1, other].isnan())
    assert y[0, 2, 0, 40] == math.inf and y[0, 3, 2, 63] == -math.inf
    w = torch.ones(D).cuda()
    a, b = torch.empty_like(y, device="cuda"), torch.empty_like(y, device="cuda")
    gdn.qk_norm_rope(x.cuda(), clean.cuda(), w, w, f.cuda(), a, b, interleaved=interleaved)
    heads = (a == b).all(-1).cpu()[0]
    want = torch.ones(4, 3, dtype=torch.bool)
    want[1, 1] = want[2, 0] = want[3, 2] = False
    assert torch.equal(heads, want)


# ---------------------------------------------------------------- the cache
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,K,Hq,Hkv,D,page,rot,norm,tree", [
    (1, 1, 16, 2, 256, 16, 64, True, False), (3, 5, 4, 2, 64, 16, 64, False, True), (2, 64, 6, 3, 128, 32, 128, True, True),
    (9, 16, 0, 1, 64, 64, 30, True, True), (2, 300, 8, 4, 64, 16, 64, True, False), (1, 70, 0, 5, 128, 1024, 0, False, False),
    (33, 2, 4, 4, 256, 128, 256, True, False)])
def test_append(B, K, Hq, Hkv, D, page, rot, norm, tree, dtype):
    say("append", B, K, Hq, Hkv, D, page, rot, norm, tree, dtype)
    g = torch.Generator().manual_seed(K + D)
    r = random.Random(B)
    lens = [r.choice([0, 1, page - 1, page, 3 * page + 5, -2]) for _ in range(B)]
    P = max(max(n, 0) + K for n in lens) // page + 1
    lens[0] = P * page - max(1, K // 2)                     # a window that runs past the table
    n_pages = B * P + 3
    ids = list(range(n_pages))
    r.shuffle(ids)
    table = [[ids[b * P + s] for s in range(P)] for b in range(B)]
    table[-1][0], table[-1][-1] = -1, n_pages               # empty slots
    count = [r.choice([0, K, K + 3, max(1, K // 2)]) for _ in range(B)]
    count[0] = K
    parent = trees(B, K, K) if tree else None
    row = randn(g, B, K, (Hq + 2 * Hkv) * D, dtype=dtype)
    wq, wk = (1 + 0.3 * torch.randn(D, generator=g) if norm and h else None for h in (Hq, Hkv))
    f = freqs_of(rot) if rot else None
    pool = randn(g, 2, n_pages, Hkv, page, D, dtype=dtype)
    dp, dr = pool.cuda(), row.cuda()

    def parts(x):
        cut = (0, Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D)
        return [x[..., a:b].unflatten(-1, ((b - a) // D, D)) if b > a else None for a, b in zip(cut, cut[1:])]

    q, k, v = parts(dr)
    qo = torch.full((B, K, Hq, D), 9.0, dtype=dtype).cuda() if Hq else None
    up = lambda w: None if w is None else w.cuda()
    kw = dict(parent=None if parent is None else dev(parent), count=dev(count))
    gdn.kv_append_rope(k, v, dp[0], dp[1], dev(lens), dev(table), up(f), q=q, q_out=qo, wq=up(wq), wk=up(wk), eps=1e-6, **kw)
    # the keys are those of the calls without a cache, bit for bit; the values byte copies
    ones = torch.ones(D).cuda()
    kt = torch.full((B, K, Hkv, D), 7.0, dtype=dtype).cuda()
    if norm:
        qt = torch.full((B, K, max(Hq, 1), D), 9.0, dtype=dtype).cuda()
        gdn.qk_norm_rope(q if Hq else k[:, :, :1], k, up(wq) if Hq else ones, up(wk), up(f), qt, kt, lens=dev(lens), **kw)
        assert not Hq or torch.equal(qo, qt)
    elif rot:
        gdn.rope(k, kt, up(f), lens=dev(lens), **kw)
        if Hq:
            qt = torch.full((B, K, Hq, D), 9.0, dtype=dtype).cuda()
            gdn.rope(q, qt, up(f), lens=dev(lens), **kw)
            assert torch.equal(qo, qt)
    else:
        kt = k
    kv_ref.append(kt.cpu(), parts(row)[2], pool[0], pool[1], lens, table, count)
    assert torch.equal(dp.cpu(), pool)
    where = ref.positions(B, K, lens=lens, parent=parent)
    there = torch.arange(K)[None] < torch.tensor(count)[:, None]
    if Hq:
        want, off = ref.turned(parts(row)[0], where, f if rot else torch.zeros(0, dtype=torch.float64), False, 1.0, wq)
        check(qo.cpu(), want, off, dtype, there)
        assert bool((qo.cpu()[~there] == 9.0).all())


def test_append_positions_of_their_own():
    """pos turns the keys; the slots still go by lens."""
    say("append pos")
    g = torch.Generator().manual_seed(8)
    B, K, H, D, page = 2, 4, 2, 64, 16
    k, v, f = randn(g, B, K, H, D, dtype=F32), randn(g, B, K, H, D, dtype=F32), freqs_of(64)
    pos = [[5, 5, 900, -3], [0, 1, 0, 1]]
    pool = torch.zeros(2, 4, H, page, D).cuda()
    gdn.kv_append_rope(k.cuda(), v.cuda(), pool[0], pool[1], dev([14, 3]), dev([[2, 0], [1, 3]]), f.cuda(), pos=dev(pos))
    want, off = ref.turned(k, pos, f)
    got = torch.stack([torch.cat([pool[0, 2, :, 14:16], pool[0, 0, :, :2]], 1), pool[0, 1, :, 3:7]]).transpose(1, 2).cpu()
    check(got, want, off, F32, torch.ones(B, K, dtype=torch.bool))
    assert torch.equal(pool[1, 1, :, 3:7].transpose(0, 1).cpu(), v[1])


def test_append_past_4_gb():
    """Pages whose offset in a plane passes 2^32 bytes."""
    say("append past 2^32")
    g = torch.Generator().manual_seed(9)
    H, D, page = 8, 256, 64
    n_pages = 2 ** 32 // (H * page * D * 2) + 2
    planes = [torch.empty(n_pages, H, page, D, dtype=BF, device="cuda") for _ in range(2)]
    k, v, f = randn(g, 1, 2, H, D, dtype=BF).cuda(), randn(g, 1, 2, H, D, dtype=BF).cuda(), freqs_of(64).cuda()
    gdn.kv_append_rope(k, v, planes[0], planes[1], dev([page - 1]), dev([[n_pages - 1, n_pages - 2]]), f)
    kt = torch.empty_like(k)
    gdn.rope(k, kt, f, lens=dev([page - 1]))
    assert torch.equal(planes[0][n_pages - 1, :, page - 1], kt[0, 0]) and torch.equal(planes[0][n_pages - 2, :, 0], kt[0, 1])
    assert torch.equal(planes[1][n_pages - 1, :, page - 1], v[0, 0]) and torch.equal(planes[1][n_pages - 2, :, 0], v[0, 1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [5, 50001])
def test_bits_that_stay(K, dtype):
    """Values, what does not turn and keys without a turn keep every bit pattern, signalling NaNs among them."""
    say("bits", K, dtype)
    g = torch.Generator().manual_seed(K)
    H, D, page, word = 4, 64, 16, torch.int16 if dtype == BF else I32
    info = torch.iinfo(word)
    bits = torch.randint(info.min, info.max + 1, (1, K, 2 * H, D), generator=g).to(word)
    bits[0, :, :, 33], bits[0, :, :, 62] = (0x7f81, -127) if dtype == BF else (0x7f800001, -8388607)   # signalling
    x = bits.view(dtype).cuda()
    k, v = x[:, :, :H], x[:, :, H:]
    P = (K + page - 1) // page
    table = torch.arange(P, dtype=I32).view(1, P).cuda()

    def rows(plane):
        return plane.cpu().view(word).transpose(1, 2).reshape(-1, H, D)[:K]

    for rot in (0, 32, 24, 22):
        pool = torch.zeros(2, P, H, page, D, dtype=dtype, device="cuda")
        gdn.kv_append_rope(k, v, pool[0], pool[1], dev([0]), table, freqs_of(rot).cuda() if rot else None)
        assert torch.equal(rows(pool[1]), bits[0, :, H:])
        assert torch.equal(rows(pool[0])[..., rot:], bits[0, :, :H, rot:])
    y = torch.empty_like(x)
    gdn.rope(x, y, freqs_of(32).cuda(), interleaved=True)
    assert torch.equal(y.cpu().view(word)[..., 32:], bits[..., 32:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode", ["pos", "lens", "chain", "tree"])
@pytest.mark.parametrize("B,K,H,D,rot", [(40, 600, 2, 64, 64), (301, 41, 3, 96, 24), (1, 9001, 1, 48, 22), (700, 13, 1, 512, 512), (5000, 3, 1, 16, 2)])
def test_many_tokens_of_few_heads(B, K, H, D, rot, mode, dtype):
    """Workgroups of many tokens, across the ends of sequences."""
    say("few heads", B, K, H, D, rot, mode, dtype)
    if mode == "tree" and K > 64:
        B, K = B * K // 50 + 1, 50
    g, r = torch.Generator().manual_seed(B), random.Random(K)
    x, f = randn(g, B, K, H, D, dtype=dtype), freqs_of(rot)
    kw = {}
    if mode == "pos":
        kw["pos"] = [[r.randint(-5000, 100000) for _ in range(K)] for _ in range(B)]
    if mode != "chain":
        kw["lens"] = [r.choice([0, -3, 77, 200000]) for _ in range(B)]
    if mode == "tree":
        kw["parent"] = trees(B, K, D)
    count = [r.choice([0, 1, K, K + 7]) for _ in range(B)]
    y = torch.full((B, K, H, D), 9.0, dtype=dtype).cuda()
    gdn.rope(x.cuda(), y, f.cuda(), count=dev(count), **{k: dev(v) for k, v in kw.items()})
    where = kw["pos"] if mode == "pos" else ref.positions(B, K, **kw)
    want, off = ref.turned(x, where, f)
    there = torch.arange(K)[None] < torch.tensor(count)[:, None]
    check(y.cpu(), want, off, dtype, there)
    assert bool((y.cpu()[~there] == 9.0).all())


def test_more_tokens_than_a_grid_has_threads():
    """2^30 tokens, of which only the last sequence's are there."""
    say("2^30 tokens")
    g = torch.Generator().manual_seed(12)
    B, K, D, page = 65535, 16384, 64, 1024
    k, v = (randn(g, 1, 1, 1, D, dtype=BF).cuda() for _ in range(2))
    f, P = freqs_of(D).cuda(), K // page
    count = torch.zeros(B, dtype=I32, device="cuda")
    count[-1] = K
    table = torch.full((B, P), -1, dtype=I32, device="cuda")
    table[-1] = torch.arange(P - 1, -1, -1, dtype=I32)
    pool = torch.zeros(2, P, 1, page, D, dtype=BF, device="cuda")
    gdn.kv_append_rope(k.expand(B, K, 1, D), v.expand(B, K, 1, D), pool[0], pool[1], torch.zeros(B, dtype=I32, device="cuda"),
                       table, f, count=count)
    want = torch.empty(1, K, 1, D, dtype=BF, device="cuda")
    gdn.rope(k.expand(1, K, 1, D), want, f)
    assert torch.equal(pool[0].flip(0).view(K, D), want.view(K, D))
    assert torch.equal(pool[1].view(K, D), v.view(1, D).expand(K, D))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,D,rot,K", [(24, 4, 256, 64, 3001), (3, 1, 64, 64, 40001), (32, 8, 128, 128, 4100), (5, 2, 64, 24, 9000)])
def test_one_call_and_many(Hq, Hkv, D, rot, K, dtype):
    """A long window in one call and in pieces: the same bits, however a launch is cut."""
    say("one call and many", Hq, Hkv, D, rot, K, dtype)
    g = torch.Generator(device="cuda").manual_seed(K)
    page = 64
    row = torch.randn(1, K, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(dtype)
    q, k, v = (x.unflatten(-1, (-1, D)) for x in row.split((Hq * D, Hkv * D, Hkv * D), -1))
    w, f = 1 + 0.2 * torch.randn(D, generator=g, device="cuda"), freqs_of(rot).cuda()
    P = K // page + 2
    table = torch.randperm(P, generator=g, device="cuda").to(I32)[None].contiguous()
    got = []
    for step in (K, 337, 29):
        pool, qo = torch.zeros(2, P, Hkv, page, D, dtype=dtype, device="cuda"), torch.zeros(1, K, Hq, D, dtype=dtype, device="cuda")
        for at in range(0, min(K, 100 * step), step):
            n = min(step, K - at)
            gdn.kv_append_rope(k[:, at:at + n], v[:, at:at + n], pool[0], pool[1], dev([at + 7]), table, f, q=q[:, at:at + n],
                               q_out=qo[:, at:at + n], wq=w, wk=w)
        got.append((pool, qo, min(K, 100 * step)))
    for pool, qo, n in got[1:]:
        assert torch.equal(qo[:, :n], got[0][1][:, :n])
        rows = torch.arange(7, n + 7, device="cuda")
        ids = table[0, rows // page].long()
        assert torch.equal(pool[:, ids, :, rows % page], got[0][0][:, ids, :, rows % page])


@pytest.mark.parametrize("interleaved", [False, True])
def test_more_than_4_gb(interleaved):
    """A window of more than 2^32 bytes: its last token is right."""
    say("rope past 2^32", interleaved)
    g = torch.Generator().manual_seed(6)
    B, K, H, D = 9, 16384, 64, 256
    x = torch.zeros(B, K, H, D, dtype=BF, device="cuda")
    last = randn(g, 1, 1, H, D, dtype=BF)
    x[-1, -1] = last[0, 0].cuda()
    f = freqs_of(64)
    gdn.rope(x, x, f.cuda(), interleaved=interleaved)
    want, off = ref.turned(last, [[K - 1]], f, interleaved)
    check(x[-1:, -1:].cpu(), want, off, BF, torch.ones(1, 1, dtype=torch.bool))
    assert float(x[:-1].abs().max()) == 0.0


def test_captured_and_on_two_streams():
    """A window's calls in a graph, replayed with other inputs in the same buffers and eager work between, and the same calls
    on two streams at once."""
    say("graph and streams")
    g = torch.Generator().manual_seed(4)
    B, K, Hq, H, D, page = 8, 7, 8, 2, 128, 16
    f = freqs_of(64).cuda()
    w = torch.ones(D).cuda()

    def state():
        return dict(q=randn(g, B, K, Hq, D, dtype=BF).cuda(), k=randn(g, B, K, H, D, dtype=BF).cuda(),
                    v=randn(g, B, K, H, D, dtype=BF).cuda(), lens=torch.randint(0, 20, (B,), generator=g).to(I32).cuda(),
                    parent=dev(trees(B, K, random.Random(int(torch.randint(0, 99, (1,), generator=g))).random())))

    def buffers():
        return dict(pool=torch.zeros(2, 2 * B, H, page, D, dtype=BF).cuda(), qo=torch.zeros(B, K, Hq, D, dtype=BF).cuda(),
                    table=torch.arange(2 * B, dtype=I32).view(B, 2).cuda())

    def call(s, b, stream=None):
        gdn.kv_append_rope(s["k"], s["v"], b["pool"][0], b["pool"][1], s["lens"], b["table"], f, q=s["q"], q_out=b["qo"], wq=w,
                           wk=w, parent=s["parent"], stream=stream)

    inputs = [state() for _ in range(4)]
    want = []
    for s in inputs:
        b = buffers()
        call(s, b)
        want.append(b)
    torch.cuda.synchronize()
    held, out = {k: v.clone() for k, v in inputs[0].items()}, buffers()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(held, out)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            call(held, out)
    for i in (1, 2, 3, 1):
        for k in held:
            held[k].copy_(inputs[i][k])
        out["pool"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["pool"], want[i]["pool"]) and torch.equal(out["qo"], want[i]["qo"])
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [buffers() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            call(inputs[i], outs[i], streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i]["pool"], want[i]["pool"]) and torch.equal(outs[i]["qo"], want[i]["qo"])
