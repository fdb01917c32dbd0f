"""GPU results of the paged cache calls against plain Python loops (kv_ref.py):
whole numbers and byte copies, so everything has to be equal."""
import random

import pytest
import torch

from speculative_verify_gdn_amd import gdn
from tests import kv_ref

pytestmark = pytest.mark.gpu
I32 = torch.int32


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


def make_pool(g, planes, n_pages, Hkv, page, D, dtype):
    return torch.randn(planes, n_pages, Hkv, page, D, generator=g).to(dtype)


def state(seed, B, P, n_pages, page, most, spare=0.0):
    """A random valid cache: lens, table (rows of P slots), ref; some full pages shared."""
    r = random.Random(seed)
    free = list(range(n_pages))
    r.shuffle(free)
    lens, table, ref = [], [], [0] * n_pages
    for b in range(B):
        n = r.randint(0, most)
        need = (n + page - 1) // page + (r.random() < spare)
        if need > P or need > len(free):
            n, need = 0, 0
        row = []
        share = min(r.randint(0, n // page), table[b - 1].index(-1) if b and -1 in table[b - 1] else 0) if b and r.random() < 0.4 else 0
        share = min(share, lens[b - 1] // page) if b else 0
        for s in range(need):
            row.append(table[b - 1][s] if s < share else free.pop())
            ref[row[-1]] += 1
        lens.append(n)
        table.append(row + [-1] * (P - need))
    return lens, table, ref


@pytest.mark.parametrize("seed,B,P,n_pages,page,most", [
    (0, 1, 3, 4, 16, 30), (1, 7, 6, 40, 16, 60), (2, 64, 9, 700, 32, 200), (3, 33, 5, 50, 64, 200),
    (4, 1500, 3, 9001, 16, 30), (5, 5, 70, 400, 16, 900), (6, 300, 4, 12000, 128, 300)])
def test_reserve(seed, B, P, n_pages, page, most):
    say("reserve", seed, B, P, n_pages, page)
    lens, table, ref = state(seed, B, P, n_pages, page, most, spare=0.3)
    r = random.Random(seed + 100)
    add = [r.choice([-1, 0, 1, 2, 5, 16, 33, page, page + 1]) for _ in range(B)]
    lens[0] = lens[0] if seed % 2 else -lens[0]
    d = [dev(x) for x in (lens, add, table, ref)]
    granted = torch.full((B,), 99, dtype=I32).cuda()
    gdn.kv_reserve(d[0], d[1], d[2], d[3], page, granted)
    want = kv_ref.reserve(lens, add, table, ref, page)
    assert granted.tolist() == want
    assert d[2].tolist() == table
    assert d[3].tolist() == ref


def test_reserve_runs_out_and_bad_ids():
    say("reserve runs out")
    table = [[5, -1, -1], [-7, 99, -1], [-1, -1, -1], [0, -1, -1]]
    ref = [1, 0, 0, 1, 0, 1]
    lens, add = [16, 0, 0, 3], [32, 20, 16, 5]     # 2, 2 (empty slots -7 and 99), 1, 0 pages; 3 are free
    d = [dev(x) for x in (lens, add, table, ref)]
    granted = dev([9] * 4)
    gdn.kv_reserve(d[0], d[1], d[2], d[3], 16, granted)
    assert kv_ref.reserve(lens, add, table, ref, 16) == granted.tolist() == [32, 0, 0, 5]
    assert d[2].tolist() == table and d[3].tolist() == ref


GEOM = [(1, 16, 64, torch.bfloat16), (2, 32, 128, torch.float32), (5, 64, 256, torch.bfloat16), (3, 128, 64, torch.float32)]


@pytest.mark.parametrize("Hkv,page,D,dtype", GEOM)
@pytest.mark.parametrize("B,K,wide,ragged", [(1, 1, 0, False), (3, 5, 16, True), (9, 64, 0, True)])
def test_append(Hkv, page, D, dtype, B, K, wide, ragged):
    say("append", Hkv, page, D, dtype, B, K, wide)
    g = torch.Generator().manual_seed(B * 7 + K)
    P, n_pages = 6, 6 * B + 2
    lens, table, ref = state(B + K, B, P, n_pages, page, 3 * page)
    lens[0] = P * page - 1                                  # the window runs past the table
    for row in table:                                       # pages under the windows; one row lacks some
        row[:] = [random.Random(K).randrange(n_pages) if p < 0 else p for p in row] if row is not table[-1] else row
    ids = list(range(n_pages))
    random.Random(1).shuffle(ids)
    for b, row in enumerate(table):                         # distinct pages: no two tokens meet
        row[:] = [ids[b * P + s] if p >= 0 else p for s, p in enumerate(row)]
    pool = make_pool(g, 2, n_pages, Hkv, page, D, dtype)
    rows = torch.randn(B, K, 2 * Hkv * D + wide, generator=g).to(dtype)
    count = [min(K, 1 + 3 * b) if b % 3 else K + 4 for b in range(B)] if ragged else None
    dp, dr = pool.cuda(), rows.cuda()
    k, v = (x[..., o:o + Hkv * D].unflatten(-1, (Hkv, D)) for x in (dr,) for o in (0, Hkv * D))
    gdn.kv_append(k, v, dp[0], dp[1], dev(lens), dev(table), count=None if count is None else dev(count))
    kc, vc = (rows[..., o:o + Hkv * D].unflatten(-1, (Hkv, D)) for o in (0, Hkv * D))
    kv_ref.append(kc, vc, pool[0], pool[1], lens, table, count)
    assert torch.equal(dp.cpu(), pool)


def test_append_refuses_uneven_tokens():
    say("append strides")
    pool = torch.zeros(2, 4, 2, 16, 64, dtype=torch.bfloat16).cuda()
    t, n = dev([[0, 1], [2, 3]]), dev([0, 0])
    k = torch.zeros(3, 2, 2, 64, dtype=torch.bfloat16).cuda().transpose(0, 1)
    with pytest.raises(ValueError):
        gdn.kv_append(k, k, pool[0], pool[1], n, t)
    k = torch.zeros(2, 3, 64, 2, dtype=torch.bfloat16).cuda().transpose(2, 3)
    with pytest.raises(ValueError):
        gdn.kv_append(k, k, pool[0], pool[1], n, t)
    with pytest.raises(TypeError):
        gdn.kv_append(k.contiguous(), k.contiguous(), pool[0], pool[1], n.long(), t)


@pytest.mark.parametrize("Hkv,page,D,dtype", GEOM)
@pytest.mark.parametrize("B,N,planes,shape", [(1, 1, 2, "chain"), (4, 7, 2, "tree"), (3, 64, 6, "tree"),
                                              (6, 32, 20, "tree"), (5, 16, 1, "chain"), (2, 33, 5, "bad")])
def test_rollback_tree(Hkv, page, D, dtype, B, N, planes, shape):
    say("rollback", Hkv, page, D, dtype, B, N, planes, shape)
    g = torch.Generator().manual_seed(N)
    r = random.Random(N * 10 + B)
    P = 130 // page + 8
    n_pages = P * B + 1
    ids = list(range(n_pages))
    r.shuffle(ids)
    lens = [r.choice([0, 1, page - 1, page, page + 3, r.randint(0, 2 * page)]) for _ in range(B)]
    table = [[ids[b * P + s] if s * page < lens[b] + N else -1 for s in range(P)] for b in range(B)]
    ref = [0] * n_pages
    for row in table:
        for p in row:
            if p >= 0:
                ref[p] = r.choice([1, 1, 2])
    parent = None
    if shape != "chain":
        parent = [[r.choice([-1, i - 1, max(i - 2, -1), r.randint(-1, i)]) if i else r.choice([-1, 0, 5]) for i in range(N)]
                  for _ in range(B)]
        if shape == "bad":
            parent[0][3], parent[0][4] = 3, N + 9           # not below the node: roots
            table[0][0], table[1][1 % P] = -1, n_pages + 3   # missing pages
    node = [r.randint(0, N - 1) for _ in range(B)]
    node[-1] = -1 if B > 1 else node[-1]
    count = [N if b % 2 else max(0, N - 2) for b in range(B)]
    pool = make_pool(g, planes, n_pages, Hkv, page, D, dtype)
    dp, dt, dr, dl = pool.cuda(), dev(table), dev(ref), dev(lens)
    out = dl if B % 2 else torch.zeros_like(dl)             # in place too
    gdn.kv_rollback_tree(dev(node), None if parent is None else dev(parent), dl, dt, dr, dp, out, count=dev(count), N=N)
    want = kv_ref.rollback(node, parent, lens, table, ref, pool, N, count)
    assert out.tolist() == want
    assert dt.tolist() == table and dr.tolist() == ref
    assert torch.equal(dp.cpu(), pool)


def test_free():
    say("free")
    lens, table, ref = state(3, 20, 300, 3000, 16, 3000)
    table[4][2] = 12345                                     # an id out of range: an empty slot
    rows = [3, 19, 3, -1, 20, 4, 0]
    d = [dev(x) for x in (rows, lens, table, ref)]
    gdn.kv_free(*d)
    kv_ref.free(rows, lens, table, ref)
    assert d[1].tolist() == lens and d[2].tolist() == table and d[3].tolist() == ref


@pytest.mark.parametrize("Hkv,page,D,dtype", GEOM)
@pytest.mark.parametrize("n,length,spare,planes", [(1, 0, 1, 2), (3, 33, 2, 4), (40, 130, 60, 2), (200, 70, 150, 1)])
def test_fork(Hkv, page, D, dtype, n, length, spare, planes):
    say("fork", Hkv, page, D, dtype, n, length, spare)
    g = torch.Generator().manual_seed(n)
    r = random.Random(n)
    P, B = 12, n + 3
    heldn = 2 * ((length + page - 1) // page)
    n_pages = heldn + spare + 2
    ids = list(range(n_pages))
    r.shuffle(ids)
    table = [[-1] * P for _ in range(B)]
    lens, ref = [0] * B, [0] * n_pages
    for b in (0, 1):                                        # two prompts, one a token shorter
        lens[b] = max(length - b, 0)
        for s in range((lens[b] + page - 1) // page):
            table[b][s] = ids.pop()
            ref[table[b][s]] = 1
    lens[2], table[2][0] = 5, ids.pop()                     # a row that still holds a page
    ref[table[2][0]] = 1
    src = [r.choice([0, 0, 1]) for _ in range(n)]
    dst = list(range(3, 3 + n))
    if n > 2:
        src[1], dst[2] = B + 5, 2                           # no such row; a full row
    pool = make_pool(g, planes, n_pages, Hkv, page, D, dtype)
    dp, dl, dt, dr = pool.cuda(), dev(lens), dev(table), dev(ref)
    granted = torch.full((n,), 7, dtype=I32).cuda()
    gdn.kv_fork(dev(src), dev(dst), dl, dt, dr, dp, granted)
    want = kv_ref.fork(src, dst, lens, table, ref, pool)
    assert granted.tolist() == want
    assert dl.tolist() == lens and dt.tolist() == table and dr.tolist() == ref
    assert torch.equal(dp.cpu(), pool)


def test_fork_of_a_row_without_its_pages():
    say("fork incomplete")
    pool = torch.randn(2, 6, 1, 16, 64).cuda()
    lens, table, ref = [40, 900, 0, 0], [[0, -1, 2], [1, 3, 4], [-1] * 3, [-1] * 3], [1, 1, 1, 1, 1, 0]
    d = dev(lens), dev(table), dev(ref)
    granted = dev([3, 3])
    before = pool.clone()
    gdn.kv_fork(dev([0, 1]), dev([2, 3]), *d, pool, granted)
    assert granted.tolist() == [0, 0]
    assert [x.tolist() for x in d] == [lens, table, ref] and torch.equal(pool, before)


@pytest.mark.parametrize("n_pages,live,Hkv,page,D,dtype,planes", [
    (1, 0, 1, 16, 64, torch.bfloat16, 1), (1, 1, 1, 16, 64, torch.bfloat16, 1), (9, 4, 3, 16, 128, torch.float32, 2),
    (301, 300, 2, 32, 64, torch.bfloat16, 3), (4097, 1500, 1, 16, 64, torch.bfloat16, 2),
    (9000, 4500, 1, 16, 64, torch.float32, 1), (64, 0, 1, 16, 64, torch.float32, 2), (120, 60, 5, 128, 256, torch.bfloat16, 2)])
def test_compact(n_pages, live, Hkv, page, D, dtype, planes):
    say("compact", n_pages, live, Hkv, page, D, dtype, planes)
    g = torch.Generator().manual_seed(n_pages)
    r = random.Random(live)
    ids = r.sample(range(n_pages), live)
    ref = [0] * n_pages
    for p in ids:
        ref[p] = r.randint(1, 3)
    rows = 7
    P = (live + rows - 1) // rows + 2
    flat = ids + [-1, -5, n_pages + 2] + ids[:3]
    flat = (flat + [-1] * (rows * P))[:rows * P]
    table = [flat[i * P:(i + 1) * P] for i in range(rows)]
    pool = make_pool(g, planes, n_pages, Hkv, page, D, dtype)
    dp, dt, dr = pool.cuda(), dev(table), dev(ref)
    t2, r2 = torch.zeros_like(dt), torch.full_like(dr, 55)
    gdn.kv_compact(dt, dr, dp, t2, r2, gdn.kv_compact_workspace(dr))
    want_t, want_r = kv_ref.compact(table, ref, pool)
    assert t2.tolist() == want_t and r2.tolist() == want_r
    assert torch.equal(dp.cpu(), pool)


@pytest.mark.parametrize("Hkv,page,D,dtype", GEOM)
@pytest.mark.parametrize("n,planes", [(0, 1), (1, 2), (3, 5), (60, 3)])
def test_copy(Hkv, page, D, dtype, n, planes):
    say("copy", Hkv, page, D, dtype, n, planes)
    g = torch.Generator().manual_seed(n)
    n_pages = 2 * n + 5
    ids = random.Random(n).sample(range(n_pages), 2 * n)
    src, dst = ids[:n], ids[n:]
    pool = make_pool(g, planes, n_pages, Hkv, page, D, dtype)
    want = pool.clone()
    if n:
        want[:, dst] = pool[:, src]
    if n > 1:
        want[:, dst[1]] = pool[:, dst[1]]
        src[1] = n_pages                                    # passed over
    dp = pool.cuda()
    gdn.kv_copy(dev(src), dev(dst), dp)
    assert torch.equal(dp.cpu(), want)


def test_offsets_past_32_bits():
    say("offsets past 32 bits")
    n_pages, Hkv, page, D = 9000, 8, 128, 256               # 4.7 GB a plane
    pool = torch.empty(2, n_pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    a, b = n_pages - 2, n_pages - 1
    pool[:, a] = torch.randn(2, Hkv, page, D, device="cuda").to(torch.bfloat16)
    pool[:, b] = 0
    gdn.kv_copy(dev([a]), dev([b]), pool)
    assert torch.equal(pool[:, a], pool[:, b])
    k = torch.randn(1, 3, Hkv, D, device="cuda").to(torch.bfloat16)
    gdn.kv_append(k, -k, pool[0], pool[1], dev([126]), dev([[a, b]]))
    assert torch.equal(pool[0, a, :, 126:].transpose(0, 1), k[0, :2]) and torch.equal(pool[1, b, :, 0], -k[0, 2])
    ref = torch.zeros(n_pages, dtype=I32, device="cuda")
    ref[a] = ref[b] = 1
    table, lens = dev([[a, b]]), dev([126])
    gdn.kv_rollback_tree(dev([2]), dev([[-1, -1, 0]]), lens, table, ref, pool, lens)
    assert lens.tolist() == [128] and table.tolist() == [[a, -1]] and int(ref[b]) == 0
    assert torch.equal(pool[0, a, :, 126:].transpose(0, 1), k[0, [0, 2]])


def test_a_window_in_a_graph_and_on_another_stream():
    """reserve, append, rollback captured and replayed, the state reset in between by eager work."""
    say("graph")
    g = torch.Generator().manual_seed(4)
    B, K, Hkv, page, D, P, n_pages = 5, 6, 2, 16, 64, 6, 40
    lens0, table0, ref0 = state(9, B, P, n_pages, page, 60)
    pool0 = make_pool(g, 4, n_pages, Hkv, page, D, torch.bfloat16)
    k, v = (torch.randn(B, K, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2))
    parent = [[i - 1 if i % 2 else i - 2 for i in range(K)] for _ in range(B)]
    node = [5, 0, -1, 3, 4]
    d = dict(lens=dev(lens0), table=dev(table0), ref=dev(ref0), pool=pool0.cuda(), granted=dev([0] * B), out=dev([0] * B),
             add=dev([K] * B), node=dev(node), parent=dev(parent), k=k.cuda(), v=v.cuda())

    def window(stream=None):
        gdn.kv_reserve(d["lens"], d["add"], d["table"], d["ref"], page, d["granted"], stream=stream)
        gdn.kv_append(d["k"], d["v"], d["pool"][2], d["pool"][3], d["lens"], d["table"], count=d["granted"], stream=stream)
        gdn.kv_rollback_tree(d["node"], d["parent"], d["lens"], d["table"], d["ref"], d["pool"], d["out"],
                             count=d["granted"], stream=stream)

    lens, table, ref, pool = list(lens0), [list(r) for r in table0], list(ref0), pool0.clone()
    granted = kv_ref.reserve(lens, [K] * B, table, ref, page)
    kv_ref.append(k, v, pool[2], pool[3], lens, table, granted)
    out = kv_ref.rollback(node, parent, lens, table, ref, pool, K, granted)

    def check():
        torch.cuda.synchronize()
        assert d["table"].tolist() == table and d["ref"].tolist() == ref and d["out"].tolist() == out
        assert torch.equal(d["pool"].cpu(), pool)

    def reset():
        d["table"].copy_(dev(table0))
        d["ref"].copy_(dev(ref0))
        d["pool"].copy_(pool0.cuda())
        d["out"].zero_()
        torch.cuda.synchronize()

    window()
    check()
    reset()
    side = torch.cuda.Stream()
    window(side)
    check()
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        window()
    for _ in range(3):
        reset()
        graph.replay()
        check()
