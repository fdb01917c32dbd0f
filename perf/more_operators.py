"""Cases that time what a verify window passes around the paged attention of a
hybrid model: its queries and keys normed, turned to their positions and put
into the cache, its logits adjusted, and its accepted node found.

Five kinds of pass, each as a serving loop makes it:

  rope    heads turned by the position of their token (pairs of the two halves,
          or neighbours; a part of the head; frequencies scaled for long contexts)
  norm    the RMS norm of every query and key head, then the same turn
  append  keys normed, turned and stored in the paged cache beside their values,
          queries normed and turned in the same pass
  logits  penalties for tokens already seen (history and drafted path), biases
          and grammar masks on the logits of every node, and the best token
  accept  the deepest drafted node whose path the best tokens confirm, and the
          history with that path appended

A window is B sequences of K tokens: a prompt (position start + t), a chain or a
draft tree given by parents (position start + depth).  A pool plane is
[n_pages][Hkv][page][D], a table row the page ids of one sequence.  With `own`
false `run` is the plain form in elementary torch operations, with `own` true
the calls of speculative_verify_gdn_amd.gdn.
"""
from __future__ import annotations

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    w = dict(Hk=0, rot=64, pairs="halves", scaled=False, dtype="bf16", tree=False, ragged=False, start=0)
    n = dict(w, norm=True, page=16, q=True)
    lg = dict(op="logits", dtype="bf16", tree=False, ragged=False, out=True, mask=False, bias=0, noise=False)
    return [
        # one token's query heads: the latency of a call
        dict(w, op="rope", name="rope one", B=1, K=1, Hq=16, D=256, start=777),
        # prompts of four sequences, whole heads of neighbouring pairs, frequencies scaled for a long context
        dict(w, op="rope", name="rope prompt", B=4, K=4096, Hq=32, D=128, rot=128, pairs="neighbours", scaled=True),
        # a verify step's window: draft trees of ragged size behind long contexts, a quarter of the head turned
        dict(n, op="norm", name="norm window", B=32, K=8, Hq=24, Hk=4, D=256, tree=True, ragged=True, start=8192),
        # an odd number of prompt tokens, fp32
        dict(n, op="norm", name="norm prompt", B=3, K=2731, Hq=32, Hk=8, D=128, rot=128, dtype="f32"),
        # the decode step of one sequence
        dict(n, op="append", name="append one", B=1, K=1, Hq=16, Hk=2, D=256, start=777),
        # 64 sequences verify draft trees of 16 nodes at far positions
        dict(n, op="append", name="append verify", B=64, K=16, Hq=24, Hk=4, D=256, page=64, tree=True, scaled=True, start=200003),
        # two prompts into the cache, no norm
        dict(n, op="append", name="append prompt", B=2, K=8192, Hq=32, Hk=8, D=128, rot=128, norm=False),
        # one sequence, one token, fp32 logits of an odd vocabulary: penalties alone
        dict(lg, name="logits one", B=1, K=1, V=50021, seen=777, dtype="f32"),
        # the batched verify window: draft trees, a grammar mask for every node, biased tokens
        dict(lg, name="logits verify", B=32, K=8, V=131072, seen=4000, tree=True, ragged=True, mask=True, bias=100),
        # 64 sequences sample a token each: temperature, and Gumbel noise added to find it
        dict(lg, name="logits sample", B=64, K=1, V=131072, seen=1500, dtype="f32", noise=True),
        # one sequence's tree of 16 nodes
        dict(op="accept", name="accept one", B=1, K=16, tree=True, ragged=False),
        # a large batch of ragged trees
        dict(op="accept", name="accept batch", B=512, K=32, tree=True, ragged=True),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["rope", "rope", "norm", "norm", "append", "append", "append", "logits", "logits", "logits", "accept"])
    c = dict(op=op, tree=rng.random() < 0.5, ragged=rng.random() < 0.4)
    if op == "accept":
        return dict(c, B=_log(rng, 1, 512), K=rng.randint(1, 32))
    c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
    c["B"] = _log(rng, 1, 64)
    if op == "logits":
        c.update(K=rng.choice([1, 1, 2, 3, 5, 8, 13, 16, 32]), V=_log(rng, 2000, 160000), seen=_log(rng, 1, 20000), out=rng.random() < 0.8,
                 mask=rng.random() < 0.5, bias=rng.choice([0, 0, 1, 17, 300]), noise=rng.random() < 0.3)
        while c["B"] * c["K"] * c["V"] * (2 if c["dtype"] == "bf16" else 4) > 7e7:
            c["B"], c["K"] = (c["B"] + 1) // 2, (c["K"] + 1) // 2
        return c
    c["tree"] = c["tree"] and rng.random() < 0.7
    c["K"] = rng.randint(1, 32) if c["tree"] else _log(rng, 1, 8192)
    Hk = rng.choice([1, 2, 4, 5, 8])
    D = rng.choice([64, 128, 256] if op == "append" else [64, 80, 96, 128, 192, 256])
    c.update(D=D, Hk=0 if op == "rope" else Hk, Hq=Hk * rng.choice([1, 2, 3, 4, 6]), rot=rng.choice([D, D, D // 2, 32]),
             pairs=rng.choice(["halves", "halves", "neighbours"]), scaled=rng.random() < 0.4, start=rng.choice([0, rng.randint(0, 1000), _log(rng, 1, 1000000)]))
    if op != "rope":
        c.update(norm=op == "norm" or rng.random() < 0.6, page=rng.choice([16, 32, 64, 128]), q=op == "norm" or rng.random() < 0.7)
    while work(c)["bytes"] > 3.5e8:
        c["B"], c["K"] = (c["B"] + 1) // 2, max(1, c["K"] * 2 // 3)
    return c


def _trees(B, N, seed):
    """Random draft trees, parents first: [B][N] int32, node 0 the root."""
    back = torch.randint(1, 4, (B, N), generator=torch.Generator().manual_seed(seed))
    parent = (torch.arange(N)[None] - back).clamp(min=0).to(torch.int32)
    parent[:, 0] = -1
    return parent


def _frequencies(rot, scaled):
    """Radians a position for each pair, and the factor on cosine and sine.  Scaled: by 8 for contexts 8 times
    as long as 32768, where a pair turns less than once over those; unchanged where it turns over 32 times;
    in between a part of each (YaRN: Peng et al. 2023)."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 1000000.0 ** (-2.0 * i / rot)
    if not scaled:
        return f.cuda(), 1.0
    turns = 32768.0 * f / (2 * math.pi)
    keep = (torch.log(turns) / math.log(32.0)).clamp(0, 1)
    return (f * keep + f / 8.0 * (1 - keep)).cuda(), float(torch.tensor(0.1 * math.log(8.0) + 1.0, dtype=torch.float32))


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    gc = torch.Generator().manual_seed(seed + 1)
    op, B, K = case["op"], case["B"], case["K"]
    s = dict(case)
    s["count"] = torch.randint(1, K + 1, (B,), generator=gc, dtype=torch.int32).to(dev) if case["ragged"] else None
    s["parent"] = _trees(B, K, seed).to(dev) if case["tree"] else None

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=dev, dtype=torch.int32)

    if op == "accept":
        V = 32000
        target = ints(0, V, B, K)
        up = s["parent"].long().clamp(min=0) if case["tree"] else (torch.arange(K, device=dev) - 1).clamp(min=0)[None].expand(B, K)
        good = torch.rand(B, K, generator=g, device=dev) < 0.75
        s.update(target=target, tokens=torch.where(good, torch.gather(target, 1, up), ints(0, V, B, K)), history=ints(0, V, B, 2048),
                 lens=ints(0, 2048, B), node=torch.zeros(B, dtype=torch.int32, device=dev), next=torch.zeros(B, dtype=torch.int32, device=dev),
                 lens_out=torch.zeros(B, dtype=torch.int32, device=dev))
        return s
    dt = _TYPES[case["dtype"]]
    if op == "logits":
        V, seen = case["V"], case["seen"]
        s["logits"] = torch.empty(B, K, V, dtype=dt, device=dev).normal_(0.0, 2.5, generator=g)
        # the history: few distinct tokens, as text has
        common = ints(0, V, B, max(1, seen // 4))
        s["history"] = torch.gather(common, 1, ints(0, common.shape[1], B, seen).long())
        s["history_lens"] = ints(seen * 3 // 4, seen + 1, B)
        s["history_start"] = (s["history_lens"] // 3).to(torch.int32)
        s["tokens"] = ints(0, V, B, K)
        # repetition, presence, frequency, temperature
        s["params"] = torch.stack([1.05 + 0.25 * torch.rand(B, generator=g, device=dev), 0.3 * torch.rand(B, generator=g, device=dev),
                                   0.2 * torch.rand(B, generator=g, device=dev), 0.6 + 0.5 * torch.rand(B, generator=g, device=dev)], 1).contiguous()
        m = case["bias"]
        s["bias_ids"] = (torch.arange(m, device=dev, dtype=torch.int32) * (V // m) + ints(0, V // m, B, m)).contiguous() if m else None
        s["bias_values"] = torch.randn(B, m, generator=g, device=dev) * 3 if m else None
        # about one token of eight is allowed
        W = (V + 31) // 32
        s["mask"] = (ints(-2**31, 2**31 - 1, B, K, W) & ints(-2**31, 2**31 - 1, B, K, W) & ints(-2**31, 2**31 - 1, B, K, W)) if case["mask"] else None
        s["noise"] = -torch.log(-torch.log(torch.rand(B, K, V, generator=g, device=dev).clamp(1e-6, 0.999999))) if case["noise"] else None
        s["out_buffer"] = torch.zeros(B, K, V, dtype=dt, device=dev) if case["out"] else None
        s["best"] = torch.zeros(B, K, dtype=torch.int32, device=dev)
        return s
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    s["freqs"], s["mscale"] = _frequencies(case["rot"], case["scaled"])
    s["lens"] = torch.randint(case["start"], case["start"] + max(1, case["start"] // 8) + 1, (B,), generator=gc, dtype=torch.int32).to(dev) \
        if case["start"] else torch.zeros(B, dtype=torch.int32, device=dev)
    heads = Hq + 2 * Hk
    row = torch.empty(B, K, heads * D, dtype=dt, device=dev).normal_(0.0, 1.5, generator=g)  # a stacked projection row a token
    s["x"] = row[..., :Hq * D].unflatten(-1, (Hq, D))
    if op == "rope":
        s["y"] = torch.zeros(B, K, Hq, D, dtype=dt, device=dev)
        return s
    s["k"], s["v"] = row[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D)), row[..., (Hq + Hk) * D:].unflatten(-1, (Hk, D))
    s["wq"], s["wk"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=dev) if case["norm"] else None for _ in range(2))
    s["q_out"] = torch.zeros(B, K, Hq, D, dtype=dt, device=dev) if case["q"] else None
    if op == "norm":
        s["k_out"] = torch.zeros(B, K, Hk, D, dtype=dt, device=dev)
        return s
    # the pages under each window, in a random order; the slots before them belong to others and stay empty here
    page = case["page"]
    first, last = s["lens"].long() // page, (s["lens"].long() + K - 1) // page
    P = int(last.max()) + 1
    slot = torch.arange(P, device=dev)[None]
    under = (slot >= first[:, None]) & (slot <= last[:, None])
    n_pages = B * ((K + page - 2) // page + 1)  # as many as the windows can touch, however they start
    table = torch.full((B, P), -1, dtype=torch.int32, device=dev)
    table[under] = torch.randperm(n_pages, generator=gc)[:int(under.sum())].to(torch.int32).to(dev)
    s.update(table=table, k_pages=torch.zeros(n_pages, Hk, page, D, dtype=dt, device=dev), v_pages=torch.zeros(n_pages, Hk, page, D, dtype=dt, device=dev))
    return s


# ---------------------------------------------------------------- the framework's calls
def _run_own(s):
    from speculative_verify_gdn_amd import gdn

    op = s["op"]
    if op == "accept":
        gdn.accept_tree(s["target"], s["tokens"], s["node"], s["next"], parent=s["parent"], count=s["count"], history=s["history"],
                        lens=s["lens"], lens_out=s["lens_out"])
        return {k: s[k] for k in ("node", "next", "history", "lens_out")}
    if op == "logits":
        if "work" not in s:
            s["work"] = gdn.logits_workspace(s["logits"])
        gdn.logits_adjust(s["logits"], out=s["out_buffer"], best=s["best"], history=s["history"], history_lens=s["history_lens"],
                          history_start=s["history_start"], tokens=s["tokens"], parent=s["parent"], count=s["count"], params=s["params"],
                          bias_ids=s["bias_ids"], bias_values=s["bias_values"], mask=s["mask"], noise=s["noise"], workspace=s["work"])
        return {"best": s["best"]} if s["out_buffer"] is None else {"best": s["best"], "out": s["out_buffer"]}
    turn = dict(parent=s["parent"], count=s["count"], interleaved=s["pairs"] == "neighbours", mscale=s["mscale"])
    if op == "rope":
        gdn.rope(s["x"], s["y"], s["freqs"], lens=s["lens"], **turn)
        return {"y": s["y"]}
    if op == "norm":
        gdn.qk_norm_rope(s["x"], s["k"], s["wq"], s["wk"], s["freqs"], s["q_out"], s["k_out"], lens=s["lens"], **turn)
        return {"q": s["q_out"], "k": s["k_out"]}
    gdn.kv_append_rope(s["k"], s["v"], s["k_pages"], s["v_pages"], s["lens"], s["table"], s["freqs"], q=s["x"] if s["q"] else None,
                       q_out=s["q_out"], wq=s["wq"] if s["q"] else None, wk=s["wk"], **turn)
    got = {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    return dict(got, q=s["q_out"]) if s["q"] else got


# ---------------------------------------------------------------- the plain forms
def _ancestors(parent, K, B, dev):
    """[B][K][K] truth: j is i or an ancestor of i."""
    i = torch.arange(K, device=dev)
    if parent is None:
        return (i[None, :] <= i[:, None])[None].expand(B, K, K)
    step = ((parent[:, :, None] == i) & (i < i[:, None])).float() + torch.eye(K, device=dev)
    return torch.linalg.matrix_power(step, K) > 0


def _there(s):
    """[B][K] truth: the token is one of its window."""
    t = torch.arange(s["K"], device="cuda")[None]
    return t < s["count"][:, None] if s["count"] is not None else (t >= 0).expand(s["B"], s["K"])


def _turned(s, x, w):
    """x [B][K][H][D] in 32 bits, normed where there is a weight, and turned."""
    B, K, half = s["B"], s["K"], s["rot"] // 2
    depth = _ancestors(s["parent"], K, B, "cuda").sum(-1) - 1 if s["parent"] is not None else torch.arange(K, device="cuda")[None].expand(B, K)
    angle = (s["lens"].long()[:, None] + depth).double()[..., None] * s["freqs"]
    c, sn = ((f(angle) * s["mscale"]).float()[:, :, None, :] for f in (torch.cos, torch.sin))
    x = x.float()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    y = x.clone()
    if s["pairs"] == "halves":
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * sn, b * c + a * sn
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * sn, b * c + a * sn
    return y


def _plain_heads(s):
    there = _there(s)[:, :, None, None]

    def out(name, x, w):
        return torch.where(there, _turned(s, x, w).to(x.dtype), s[name])

    if s["op"] == "rope":
        return {"y": out("y", s["x"], None)}
    if s["op"] == "norm":
        return {"q": out("q_out", s["x"], s["wq"]), "k": out("k_out", s["k"], s["wk"])}
    at = s["lens"].long()[:, None] + torch.arange(s["K"], device="cuda")
    pick = _there(s).reshape(-1).nonzero()[:, 0] if s["count"] is not None else slice(None)
    ids, rows = torch.gather(s["table"].long(), 1, at // s["page"]).view(-1)[pick], (at % s["page"]).view(-1)[pick]
    k = _turned(s, s["k"], s["wk"]).to(s["k"].dtype)
    s["k_pages"][ids, :, rows] = k.flatten(0, 1)[pick]
    s["v_pages"][ids, :, rows] = s["v"].flatten(0, 1)[pick]
    got = {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    return dict(got, q=out("q_out", s["x"], s["wq"])) if s["q"] else got


def _counts(ids, valid, V):
    """How often each of V tokens stands among ids[...][n], where valid."""
    into = torch.where(valid, ids.long(), V)
    return torch.zeros(*ids.shape[:-1], V + 1, dtype=torch.int32, device=ids.device).scatter_add_(-1, into, torch.ones_like(into, dtype=torch.int32))[..., :V]


def _plain_logits(s):
    x = s["logits"].float()
    B, K, V = x.shape
    i = torch.arange(s["seen"], device="cuda")[None]
    past = i < s["history_lens"][:, None]
    path = _counts(s["tokens"][:, None, :].expand(B, K, K), _ancestors(s["parent"], K, B, "cuda"), V)
    seen = _counts(s["history"], past, V)[:, None] + path
    written = _counts(s["history"], past & (i >= s["history_start"][:, None]), V)[:, None] + path
    rep, presence, frequency, temp = (s["params"][:, None, None, j] for j in range(4))
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - frequency * written.float() - presence * (written > 0).float()
    if s["bias_ids"] is not None:
        x = x + torch.zeros(B, V, device="cuda").scatter_(1, s["bias_ids"].long(), s["bias_values"])[:, None]
    if s["mask"] is not None:
        v = torch.arange(V, device="cuda")
        x = torch.where((s["mask"][..., v // 32] >> (v % 32)) & 1 > 0, x, -math.inf)
    x = x / temp
    score = x if s["noise"] is None else x + s["noise"]
    top = score.amax(-1, keepdim=True)
    best = torch.where(score == top, torch.arange(V, device="cuda", dtype=torch.int32), V).amin(-1).to(torch.int32)
    best = torch.where(top[..., 0] > -math.inf, best, -1)
    there = _there(s)
    best = torch.where(there, best, 0)
    if s["out_buffer"] is None:
        return {"best": best}
    return {"best": best, "out": torch.where(there[..., None], x.to(s["logits"].dtype), s["out_buffer"])}


def _plain_accept(s):
    target, tokens, lens = s["target"], s["tokens"], s["lens"].long()
    B, K = target.shape
    i = torch.arange(K, device="cuda")[None]
    up = s["parent"].long() if s["parent"] is not None else (i - 1).expand(B, K)
    root = (up < 0) | (up >= i)
    good = (root | (tokens == torch.gather(target, 1, torch.where(root, 0, up)))) & _there(s)
    above = _ancestors(s["parent"], K, B, "cuda")
    kept = (above & ~good[:, None, :]).sum(-1) == 0
    depth = above.sum(-1)
    node = torch.where(kept, depth * K + (K - 1 - i), -1)
    some = node.amax(-1) >= 0
    node = torch.where(some, torch.argmax(node, -1), -1)
    path = torch.gather(above, 1, node.clamp(min=0)[:, None, None].expand(B, 1, K))[:, 0] & some[:, None]
    s["next"].copy_(torch.where(some, torch.gather(target, 1, node.clamp(min=0)[:, None])[:, 0], -1))
    s["node"].copy_(node)
    n = s["history"].shape[1]
    at = lens[:, None] + path.cumsum(-1) - 1
    pick = (path & (at < n)).view(-1).nonzero()[:, 0]
    s["history"][torch.arange(B, device="cuda")[:, None].expand(B, K).reshape(-1)[pick], at.view(-1)[pick]] = tokens.view(-1)[pick]
    s["lens_out"].copy_((lens + path.sum(-1)).clamp(max=n))
    return {k: s[k] for k in ("node", "next", "history", "lens_out")}


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "accept":
        return _plain_accept(state)
    return _plain_logits(state) if state["op"] == "logits" else _plain_heads(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    es = 2 if case.get("dtype") == "bf16" else 4
    op, B, K = case["op"], case["B"], case["K"]
    tokens = B * ((K + 1) / 2 if case["ragged"] else K)
    ids = B * K * 4 * case["tree"] + B * 8
    if op == "accept":
        return {"bytes": 8 * tokens + ids + 16 * B + 4 * B * 3, "flops": 0}
    if op == "logits":
        V = case["V"]
        each = es + es * case["out"] + 4 * case["noise"] + case["mask"] / 8
        return {"bytes": tokens * (V * each + 8) + B * (4 * case["seen"] + 8 * case["bias"] + 24) + ids, "flops": tokens * V}
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    heads = Hq if op == "rope" else Hq + Hk if op == "norm" else Hq * case["q"] + 2 * Hk
    per = 3.0 * case["rot"] / D + (4 if op != "rope" and case["norm"] else 0)
    return {"bytes": 2.0 * tokens * heads * D * es + ids + 4 * case["rot"], "flops": tokens * (heads - Hk * (op == "append")) * D * per}


# ---------------------------------------------------------------- the definition, in 64 bits
def _up(parent, i):
    """The nodes from the root to i; parent None: a chain."""
    path = [i]
    while True:
        p = path[-1] - 1 if parent is None else parent[path[-1]]
        if not 0 <= p < path[-1]:
            return path[::-1]
        path.append(p)


def _exact_head(s, x, w):
    """Every pair of a head as a complex number, multiplied by mscale * e^{i position frequency}."""
    B, K = s["B"], s["K"]
    if s["parent"] is None:
        depth = [list(range(K))] * B
    else:
        depth = [[len(_up(p, i)) - 1 for i in range(K)] for p in s["parent"].tolist()]
    pos = torch.tensor(depth, dtype=torch.float64, device="cuda") + s["lens"].double()[:, None]
    z = torch.polar(torch.full((), s["mscale"], dtype=torch.float64, device="cuda"), pos[..., None] * s["freqs"])[:, :, None, :]
    y = x.double()
    if w is not None:
        y = y * torch.rsqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + 1e-6) * w.double()
    half = s["rot"] // 2
    head, rest = y[..., :2 * half], y[..., 2 * half:]
    pair = head.unflatten(-1, (2, half)).transpose(-1, -2) if s["pairs"] == "halves" else head.unflatten(-1, (half, 2))
    pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
    head = (pair.transpose(-1, -2) if s["pairs"] == "halves" else pair).flatten(-2)
    return torch.cat([head, rest], -1)


def _exact_heads(s):
    B, K = s["B"], s["K"]
    count = [K] * B if s["count"] is None else s["count"].tolist()

    def out(name, x, w):
        y, to = _exact_head(s, x, w), s[name].double()
        for b, n in enumerate(count):
            to[b, :n] = y[b, :n]
        return to

    if s["op"] == "rope":
        return {"y": out("y", s["x"], None)}
    if s["op"] == "norm":
        return {"q": out("q_out", s["x"], s["wq"]), "k": out("k_out", s["k"], s["wk"])}
    k, kp, vp, page = _exact_head(s, s["k"], s["wk"]), s["k_pages"].double(), s["v_pages"].double(), s["page"]
    for b, start in enumerate(s["lens"].tolist()):
        row, t = s["table"][b].tolist(), 0
        while t < count[b]:  # the tokens of one page
            slot, at = divmod(start + t, page)
            n = min(page - at, count[b] - t)
            kp[row[slot], :, at:at + n], vp[row[slot], :, at:at + n] = k[b, t:t + n].transpose(0, 1), s["v"][b, t:t + n].transpose(0, 1).double()
            t += n
    got = {"k_pages": kp, "v_pages": vp}
    return dict(got, q=out("q_out", s["x"], s["wq"])) if s["q"] else got


def _exact_logits(s):
    if s["out_buffer"] is None:
        return None
    out, tokens = s["out_buffer"].double(), s["tokens"].tolist()
    B, K, V = out.shape
    count = [K] * B if s["count"] is None else s["count"].tolist()
    lens, start = s["history_lens"].tolist(), s["history_start"].tolist()
    for b in range(B):
        rep, presence, frequency, temp = s["params"][b].double().tolist()
        parent = None if s["parent"] is None else s["parent"][b].tolist()
        past = torch.bincount(s["history"][b, :start[b]].long(), minlength=V)
        since = torch.bincount(s["history"][b, start[b]:lens[b]].long(), minlength=V)
        for t in range(count[b]):
            n = since.clone()
            for j in _up(parent, t):
                n[tokens[b][j]] += 1
            x = s["logits"][b, t].double()
            x = torch.where(past + n > 0, x * torch.where(x > 0, 1.0 / rep, rep), x) - n * frequency - (n > 0) * presence
            if s["bias_ids"] is not None:
                x[s["bias_ids"][b].long()] += s["bias_values"][b].double()
            if s["mask"] is not None:
                bits = s["mask"][b, t].view(torch.uint8)
                allowed = torch.stack([(bits >> j) & 1 for j in range(8)], -1).view(-1)[:V] > 0
                x = x.masked_fill(~allowed, -math.inf)
            out[b, t] = x / temp
    return {"best": None, "out": out}  # (the best of nearly equal ones goes by their rounding)


def _exact_accept(s):
    target, tokens, history, lens = s["target"].tolist(), s["tokens"].tolist(), s["history"].tolist(), s["lens"].tolist()
    B, K = s["B"], s["K"]
    count = [K] * B if s["count"] is None else s["count"].tolist()
    nodes, nexts, after = [], [], []
    for b in range(B):
        parent = None if s["parent"] is None else s["parent"][b].tolist()
        best = []
        for i in range(count[b]):
            path = _up(parent, i)
            if all(tokens[b][j] == target[b][p] for p, j in zip(path, path[1:])) and len(path) > len(best):
                best = path
        nodes.append(best[-1] if best else -1)
        nexts.append(target[b][best[-1]] if best else -1)
        room = history[b]
        for i, j in enumerate(best):
            if lens[b] + i < len(room):
                room[lens[b] + i] = tokens[b][j]
        after.append(min(lens[b] + len(best), len(room)))
    return {"node": torch.tensor(nodes), "next": torch.tensor(nexts), "history": torch.tensor(history), "lens_out": torch.tensor(after)}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "accept":
        return _exact_accept(s)
    return _exact_logits(s) if s["op"] == "logits" else _exact_heads(s)
