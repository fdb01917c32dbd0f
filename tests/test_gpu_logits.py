"""The logits and acceptance calls on the GPU against the plain forms of
window_ref.py."""
import math
import random

import pytest
import torch

from speculative_verify_gdn_amd import gdn
from tests import window_ref as ref
from tests.test_gpu_rope import _gpu, dev, say, trees  # noqa: F401

pytestmark = pytest.mark.gpu
I32, BF, F32 = torch.int32, torch.bfloat16, torch.float32


def case(seed, B, K, V, seen, dtype, tree=False, ragged=False, n_bias=0, mask=False, noise=False, start=True, params=True):
    g, r = torch.Generator().manual_seed(seed), random.Random(seed)
    c = dict(x=(torch.randn(B, K, V, generator=g) * 3).to(dtype))
    if seen:
        c["history"] = torch.randint(-2, V + 2, (B, seen), generator=g).to(I32)      # some outside the vocabulary
        c["history"][:, :seen // 2] = c["history"][:, :1]                            # and one that stands there often
        c["lens"] = torch.tensor([r.choice([seen, seen // 2, 0, seen + 5, -1]) if b else seen for b in range(B)], dtype=I32)
        if start:
            c["start"] = torch.tensor([r.choice([0, -4, seen // 3, seen, seen + 1]) for _ in range(B)], dtype=I32)
    c["tokens"] = torch.randint(-1, V + 1, (B, K), generator=g).to(I32)
    c["tokens"][:, K // 2:] = c["tokens"][:, :1]                                     # the same token twice on a path
    if tree:
        c["parent"] = torch.tensor(trees(B, K, seed), dtype=I32)
    if params:
        c["params"] = torch.stack([0.7 + torch.rand(B, generator=g), torch.randn(B, generator=g), torch.randn(B, generator=g) * 0.3,
                                   0.3 + torch.rand(B, generator=g)], 1)
    if n_bias:
        c["ids"] = torch.randint(-1, V + 1, (B, n_bias), generator=g).to(I32)
        c["ids"][:, -1] = c["ids"][:, 0]                                             # an id named twice
        c["values"] = torch.randn(B, n_bias, generator=g) * 4
    if mask:
        c["mask"] = torch.randint(-2 ** 31, 2 ** 31, (B, K, (V + 31) // 32), generator=g).to(I32)
        c["mask"][0, 0] = 0                                                          # a row that allows nothing
    if noise:
        c["noise"] = -torch.log(-torch.log(torch.rand(B, K, V, generator=g).clamp(1e-6, 1 - 1e-6)))
    if ragged:
        c["count"] = torch.tensor([r.choice([0, 1, K, K + 1]) if b else K for b in range(B)], dtype=I32)
    return c


NAMES = dict(history="history", lens="history_lens", start="history_start", tokens="tokens", parent="parent", count="count",
             params="params", ids="bias_ids", values="bias_values", mask="mask", noise="noise")


def run(c, out_dtype=None, best=True, x=None, out=None):
    x = c["x"].cuda() if x is None else x
    B, K, V = x.shape
    if out is None and out_dtype is not None:
        out = torch.full((B, K, V), 9.0, dtype=out_dtype).cuda()
    b = torch.full((B, K), -7, dtype=I32).cuda() if best else None
    gdn.logits_adjust(x, out=out, best=b, workspace=gdn.logits_workspace(x) if best else None,
                      **{NAMES[k]: v.cuda() for k, v in c.items() if k in NAMES})
    return out, b


def expect(c):
    return ref.logits(c["x"], *(c.get(k) for k in "history lens start tokens parent params ids values mask count".split()))


def check(c, out, b, out_dtype):
    want, f32 = expect(c)
    there = ~want[..., 0].isnan() if not bool(c["x"].isnan().any()) else torch.ones(c["x"].shape[:2], dtype=torch.bool)
    if out is not None:
        got = out.cpu()
        # every step is one rounding in a stated order: the same bits as the plain steps in 32
        assert torch.equal(got[there], f32.to(out_dtype)[there])
        assert bool((got[~there] == 9.0).all())
        # and against 64 bits: up to five roundings of what was added up, and the output's own
        size = 8 * (c["x"].double().abs() + 8) / (0.3 if c.get("params") is not None else 1)
        finite = want.isfinite() & there[..., None]
        d = (got.double() - want).abs() / ref.rounded(5 * ref.H24 * size, want, out_dtype)
        assert float(torch.where(finite, d, 0.0).max()) <= 1.0
    if b is not None:
        score = f32 if c.get("noise") is None else f32 + c["noise"]
        assert torch.equal(b.cpu()[there], ref.best(score)[there])
        assert bool((b.cpu()[~there] == -7).all())


@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("B,K,V,seen", [(1, 1, 1, 3), (1, 1, 7, 0), (2, 3, 33, 50), (3, 16, 1000, 200), (2, 2, 4097, 30), (1, 64, 513, 100),
                                        (5, 1, 9999, 1000)])
def test_adjust(B, K, V, seen, dtype, out_dtype):
    say("logits", B, K, V, seen, dtype, out_dtype)
    for seed, kw in enumerate([dict(), dict(tree=True, ragged=True, n_bias=5, mask=True), dict(n_bias=1, noise=True, start=False),
                               dict(params=False, mask=True, noise=True), dict(tree=True, noise=True, mask=True, n_bias=40)]):
        c = case(seed * 100 + V, B, K, V, seen, dtype, **kw)
        check(c, *run(c, out_dtype), out_dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_adjust_a_large_vocabulary(dtype):
    say("logits large", dtype)
    c = case(5, 3, 4, 131072 + 3, 3000, dtype, tree=True, ragged=True, n_bias=300, mask=True)
    check(c, *run(c, dtype), dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [dict(tree=True, ragged=True, n_bias=40, mask=True, noise=True), dict(n_bias=256), dict(params=False)])
def test_adjust_in_large_slices(kw, dtype):
    """Enough rows that a workgroup takes 8192 tokens of the vocabulary, and one that ends inside a slice."""
    say("logits large slices", kw, dtype)
    c = case(11, 5, 8, 100003, 150, dtype, **kw)
    check(c, *run(c, dtype), dtype)


@pytest.mark.parametrize("capacity,seen,n_bias", [(16000, 16000, 3), (16001, 16001, 3), (20000, 700, 0), (20000, 20000, 257), (3, 3, 0), (5, 4, 257),
                                                  (1030, 1029, 1), (4, 4, 256)])
def test_texts_of_every_length(capacity, seen, n_bias):
    """Counts of 16 bits and of 32, on both sides of where they change, one token for nearly all of a text; texts that
    end inside a read of four; biases listed and not."""
    say("logits texts", capacity, seen, n_bias)
    c = case(12, 2, 2, 5000, capacity, F32, n_bias=n_bias)
    c["history"][:, :capacity - 1] = torch.tensor([[17], [4999]], dtype=I32)
    c["lens"] = torch.tensor([seen, seen - 1], dtype=I32)
    c["start"] = torch.tensor([1, seen // 2], dtype=I32)
    c["tokens"][:] = 17
    if n_bias:
        c["ids"][:, 0] = 17
    check(c, *run(c, F32), F32)


def test_logits_past_2_31():
    """More than 2^31 logits: the last row is right, and the first."""
    say("logits past 2^31")
    B, K, V = 257, 64, 131072
    x = torch.zeros(B, K, V, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(1)
    rows = torch.randn(2, V, generator=g).to(BF)
    x[0, 0], x[-1, -1] = rows[0].cuda(), rows[1].cuda()
    params = torch.tensor([1.0, 0.0, 0.0, 0.5]).repeat(B, 1).cuda()
    best = torch.empty(B, K, dtype=I32, device="cuda")
    gdn.logits_adjust(x, out=x, best=best, params=params, workspace=gdn.logits_workspace(x))
    assert torch.equal(x[0, 0].cpu(), (rows[0].float() * 2).to(BF)) and torch.equal(x[-1, -1].cpu(), (rows[1].float() * 2).to(BF))
    assert best[0, 0].item() == ref.best(rows[:1].float())[0].item() and best[-1, -1].item() == ref.best(rows[1:].float())[0].item()
    assert int(best[100, 7]) == 0 and float(x[100, 7].abs().max()) == 0.0


@pytest.mark.parametrize("B,K,V", [(64, 8, 9000), (65, 8, 9000), (33, 64, 2500), (5, 64, 33000), (64, 3, 2048), (1, 64, 140000)])
@pytest.mark.parametrize("counts", ["any", "none", "last", "one"])
def test_windows_of_every_length(B, K, V, counts):
    """Which rows a workgroup takes goes by the windows' lengths: every row that is there is right, no other is touched."""
    say("windows", B, K, V, counts)
    r = random.Random(B * K)
    c = case(B, B, K, V, 20, BF, tree=True, mask=False)
    c["count"] = torch.tensor({"any": [r.randint(-1, K + 1) for _ in range(B)], "none": [0] * B, "last": [0] * (B - 1) + [K],
                               "one": [1] * B}[counts], dtype=I32)
    out, b = run(c, BF)
    del c["params"]                                      # (the adjusting itself is tested above)
    plain, pb = run({k: v for k, v in c.items() if k != "count"}, BF)
    there = torch.arange(K)[None] < c["count"][:, None]
    assert bool((out.cpu()[~there] == 9.0).all()) and bool((b.cpu()[~there] == -7).all())
    assert not bool((out.cpu()[there] == 9.0).all(-1).any()) and bool((b.cpu()[there] >= 0).all())
    out, b = run(c, BF)
    assert torch.equal(out.cpu()[there], plain.cpu()[there]) and torch.equal(b.cpu()[there], pb.cpu()[there])
    assert bool((out.cpu()[~there] == 9.0).all()) and bool((b.cpu()[~there] == -7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("V,length,capacity,often", [
    (100, 16001, 16001, [(7, 16001)]), (9000, 33000, 40000, [(8191, 16000), (8192, 17000)]), (5000, 40000, 1 << 17, [(2047, 39990)]),
    (50, 120000, 120000, [(3, 16200), (4, 16300), (10, 40000), (49, 16255)]), (300, 900, 1 << 20, [(5, 800)]),
    (40, 100000, 383872, [(0, 50000), (1, 50000)]), (40, 100000, 383873, [(0, 50000), (1, 50000)]),
    (128, 383872, 383872, [(i, 2999) for i in range(128)]), (128, 383872, 383872, [(127 - i, 3022) for i in range(127)])])
def test_tokens_that_stand_often(V, length, capacity, often, few, dtype):
    """Long texts, tokens that stand in them more often than 14 bits count, with drafts and biases of the same ones."""
    say("often", V, length, capacity, often, few, dtype)
    g = torch.Generator().manual_seed(length)
    B, K = (2, 3) if few else (6, 64)
    c = case(1, B, K, V, 4, dtype, n_bias=3)
    text = torch.randint(0, V, (length,), generator=g).to(I32)
    at, i = torch.randperm(length, generator=g), 0
    for token, n in often:
        text[at[i:i + n]] = token
        i += n
    c["history"] = torch.zeros(B, capacity, dtype=I32)
    c["history"][:, :length] = text
    c["lens"] = torch.tensor([length, length - 1] * (B // 2), dtype=I32)
    c["start"] = torch.tensor([0, length // 3] * (B // 2), dtype=I32)
    c["tokens"][:] = often[0][0]
    c["ids"][:, 1] = often[-1][0]
    c["params"][:, 2] = torch.tensor([1e-4, -3e-5] * (B // 2))
    out, b = run(c, F32)
    # (the counts by torch, in place of the loops over texts)
    want = c["x"].float()
    for s in range(B):
        n = int(c["lens"][s])
        seen, since = (torch.bincount(c["history"][s, i:n].long(), minlength=V) for i in (0, int(c["start"][s])))
        rep, presence, frequency, temp = c["params"][s]
        for t in range(K):
            path = torch.zeros(V, dtype=torch.int64)
            path[often[0][0]] = t + 1
            x = want[s, t]
            x = torch.where(seen + path > 0, x * torch.where(x > 0, 1.0 / rep, rep), x)
            x = torch.where(since + path > 0, x - (frequency * (since + path).float() + presence), x)
            for i, v in {int(i): v for i, v in zip(c["ids"][s], c["values"][s]) if 0 <= i < V}.items():
                x[i] += v
            want[s, t] = x * (1.0 / temp)
    assert torch.equal(out.cpu(), want)
    assert torch.equal(b.cpu(), ref.best(want))


@pytest.mark.parametrize("B,K,V,n_bias", [(2, 5, 300, 256), (1, 16, 70, 256), (3, 2, 300, 257), (2, 9, 9000, 200), (2, 5, 300, 512), (3, 2, 300, 513)])
def test_biases_of_many_tokens(B, K, V, n_bias):
    """Most tokens have a bias, many ids are named twice or more, and the drafted tokens and the text's have one too."""
    say("biases", B, K, V, n_bias)
    for seed in range(4):
        c = case(seed, B, K, V, 90, F32, tree=bool(seed & 1), n_bias=n_bias)
        c["ids"][:, ::3] = torch.randint(0, min(V, 40), c["ids"][:, ::3].shape).to(I32)
        c["tokens"] = c["ids"][:, torch.arange(K) % n_bias].clone()
        c["history"][:, ::2] = c["ids"][:, torch.arange(45) % n_bias]
        out, b = run(c, F32)
        check(c, out, b, F32)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_of_the_outputs_and_in_place(dtype):
    say("logits outputs", dtype)
    c = case(6, 2, 3, 1234, 60, dtype, n_bias=4)
    out, b = run(c, dtype)
    alone, none = run(c, dtype, best=False)
    assert none is None and torch.equal(alone, out)
    none, alone = run(c)
    assert none is None and torch.equal(alone, b)
    x = c["x"].cuda()
    run(c, best=False, x=x, out=x)
    assert torch.equal(x, out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,wide,at", [(1000, 1000, 0), (1001, 1001, 0), (997, 1024, 0), (1003, 1021, 8), (4099, 5000, 16)])
def test_rows_that_start_anywhere(V, wide, at, dtype):
    """Rows at any element: slices of wider ones, odd lengths; what lies between them stays."""
    say("logits rows", V, wide, at, dtype)
    c = case(7, 2, 3, V, 50, dtype, n_bias=3, mask=True)
    rows = torch.full((2, 3, wide + at), 5.0, dtype=dtype).cuda()
    outs = torch.full((2, 3, wide + at), 5.0, dtype=dtype).cuda()
    x, out = rows[..., at:at + V], outs[..., at:at + V]
    x.copy_(c["x"])
    out.fill_(9.0)
    out, b = run(c, x=x, out=out)
    check(c, out, b, dtype)
    assert bool((outs[..., :at] == 5.0).all()) and bool((outs[..., at + V:] == 5.0).all())


def test_values_that_are_not_finite():
    """NaN is kept and never the best; infinities follow the formula; of equal ones the lowest is the best."""
    say("logits not finite")
    c = case(8, 2, 2, 700, 0, F32, params=False)
    x = c["x"]
    x[0, 0, 5], x[0, 0, 600], x[0, 0, 601] = math.nan, math.inf, math.inf
    x[0, 1] = math.nan
    x[1, 0] = -math.inf
    x[1, 1] = 2.5
    out, b = run(c, F32)
    assert torch.equal(b.cpu(), torch.tensor([[600, -1], [-1, 0]], dtype=I32))
    assert bool(((out.cpu() == x) | x.isnan()).all()) and bool(out.cpu()[0, 1].isnan().all())
    for v in (3, 511, 512, 699):                            # equal ones on both sides of a slice
        x[1, 1] = 2.5
        x[1, 1, v:] = 7.0
        assert int(run(c)[1][1, 1]) == v


def test_parameters_at_their_edges():
    say("logits parameters")
    c = case(9, 4, 2, 300, 40, F32)
    c["params"] = torch.tensor([[1.0, 0.0, 0.0, 1.0], [1.0, 0.0, 0.0, 0.0], [2.0, -1.0, 0.5, -3.0], [0.5, 0.1, math.inf, math.nan]])
    out, b = run(c, F32)
    assert torch.equal(out[0].cpu(), c["x"][0]) and torch.equal(out[1].cpu(), c["x"][1])
    c["params"][3, 3] = 0.0                                  # (a temperature that is no number counts as none)
    f32 = expect(c)[1]
    assert torch.equal(out.cpu(), f32)


def test_logits_captured_and_on_two_streams():
    say("logits graph and streams")
    cases = [case(20 + i, 4, 5, 5000, 300, BF, tree=True, n_bias=9, mask=True) for i in range(4)]
    want = [run(c, BF) for c in cases]
    keys = [k for k in cases[0] if k in NAMES]

    def held(c):
        s = {k: c[k].cuda() for k in keys}
        s.update(x=c["x"].cuda(), out=torch.zeros(4, 5, 5000, dtype=BF).cuda(), best=torch.zeros(4, 5, dtype=I32).cuda(),
                 node=torch.zeros(4, dtype=I32).cuda(), next=torch.zeros(4, dtype=I32).cuda())
        s["work"] = gdn.logits_workspace(s["x"])
        return s

    def call(s, stream=None):
        gdn.logits_adjust(s["x"], out=s["out"], best=s["best"], workspace=s["work"], stream=stream, **{NAMES[k]: s[k] for k in keys})
        gdn.accept_tree(s["best"], s["tokens"], s["node"], s["next"], parent=s["parent"], stream=stream)

    h, graph, side = held(cases[0]), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call(h)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            call(h)
    for i in (1, 2, 3, 1):
        for k in keys + ["x"]:
            h[k].copy_(cases[i][k])
        h["work"].fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h["out"], want[i][0]) and torch.equal(h["best"], want[i][1])
        nodes, nexts, _, _ = ref.accept(want[i][1].tolist(), cases[i]["tokens"].tolist(), cases[i]["parent"].tolist())
        assert h["node"].tolist() == nodes and h["next"].tolist() == nexts
    both, streams = [held(c) for c in cases[:2]], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, st in zip(both, streams):
            call(s, st)
    torch.cuda.synchronize()
    for i, s in enumerate(both):
        assert torch.equal(s["out"], want[i][0]) and torch.equal(s["best"], want[i][1])


@pytest.mark.parametrize("B,K,tree,ragged,rooted", [(1, 1, False, False, False), (1, 16, True, False, False), (7, 64, True, True, True),
                                                    (130, 33, True, True, False), (66, 5, False, True, True), (1000, 32, True, True, True)])
def test_accept(B, K, tree, ragged, rooted):
    say("accept", B, K, tree, ragged, rooted)
    r = random.Random(B + K)
    parent = trees(B, K, K) if tree else None
    target = [[r.randint(-1, 3) for _ in range(K)] for _ in range(B)]
    tokens = [[r.randint(-1, 3) for _ in range(K)] for _ in range(B)]
    for b in range(B):                                       # long paths among the short ones
        for i in range(1, K):
            p = parent[b][i] if tree else i - 1
            if 0 <= p < i and r.random() < 0.8:
                tokens[b][i] = target[b][p]
    count = [r.choice([-1, 0, 1, K, K + 2, max(1, K // 2)]) for _ in range(B)] if ragged else None
    root = [r.choice([-1, -5, 0, 1, 2]) for _ in range(B)] if rooted else None
    cap = 40
    history = [[r.randint(0, 9) for _ in range(cap)] for _ in range(B)]
    lens = [r.choice([0, 5, cap - 2, cap, cap + 9, -3]) for _ in range(B)]
    want = ref.accept(target, tokens, parent, count, root, history, lens)
    node, nxt, out = (torch.full((B,), 77, dtype=I32).cuda() for _ in range(3))
    opt = lambda v: None if v is None else dev(v)
    h, n = dev(history), dev(lens)
    kw = dict(parent=opt(parent), count=opt(count), root=opt(root))
    gdn.accept_tree(dev(target), dev(tokens), node, nxt, **kw)
    assert node.tolist() == want[0] and nxt.tolist() == want[1]
    gdn.accept_tree(dev(target), dev(tokens), node, nxt, history=h, lens=n, lens_out=out, **kw)
    assert node.tolist() == want[0] and nxt.tolist() == want[1]
    assert h.tolist() == want[2] and out.tolist() == want[3]
    h = dev(history)
    gdn.accept_tree(dev(target), dev(tokens), node, nxt, history=h, lens=n, lens_out=n, **kw)
    assert h.tolist() == want[2] and n.tolist() == want[3]
