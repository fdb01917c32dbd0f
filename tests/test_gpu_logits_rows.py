"""Workgroups of the logits call that take several rows of a window: a row's drafted
tokens are counted for it and taken back before the next one, in each of the ways
the counts are kept."""
import random

import pytest
import torch

from speculative_verify_gdn_amd import gdn
from tests import window_ref as ref
from tests.test_gpu_logits import case, run
from tests.test_gpu_rope import _gpu, say  # noqa: F401

pytestmark = pytest.mark.gpu
I32, BF, F32 = torch.int32, torch.bfloat16, torch.float32
ROWS = (33, 64, 2500)


def ancestors(parent, K):
    """[K][K]: which nodes stand on the path to each (parent None: a chain)."""
    on = torch.zeros(K, K, dtype=torch.bool)
    for t in range(K):
        up = t - 1 if parent is None else int(parent[t])
        if 0 <= up < t:
            on[t] = on[up]
        on[t, t] = True
    return on


def counts(tokens, V):
    """How often each token below V stands in a list."""
    tokens = tokens[(tokens >= 0) & (tokens < V)].long()
    return torch.bincount(tokens, minlength=V)


def expect(c):
    """The adjusted logits [B][K][V], each step rounded once in float32."""
    B, K, V = c["x"].shape
    want = c["x"].to(F32, copy=True)
    for b in range(B):
        n = min(max(int(c["lens"][b]), 0), c["history"].shape[1])
        first = min(max(int(c["start"][b]), 0), n)
        text = c["history"][b, :n]
        seen, since = counts(text, V), counts(text[first:], V)
        on = ancestors(c["parent"][b] if "parent" in c else None, K)
        rep, presence, frequency, temp = c["params"][b]
        bias = {int(v): float(f) for v, f in zip(c["ids"][b], c["values"][b]) if 0 <= v < V}
        at, by = torch.tensor(list(bias), dtype=torch.int64), torch.tensor(list(bias.values()), dtype=F32)
        for t in range(K):
            path = counts(c["tokens"][b][on[t]], V)
            x = want[b, t]
            x = torch.where(seen + path > 0, x * torch.where(x > 0, 1.0 / rep, rep), x)
            x = torch.where(since + path > 0, x - (frequency * (since + path).float() + presence), x)
            x[at] += by
            want[b, t] = x * (1.0 / temp)
    return want


def several(seed, B, K, V, dtype, capacity, n_bias, tree):
    """Drafted tokens that repeat on paths and between branches, that have biases, and that stand in the text."""
    g, r = torch.Generator().manual_seed(seed), random.Random(seed)
    c = case(seed, B, K, V, capacity, dtype, tree=tree, n_bias=n_bias)
    if tree:                                                     # siblings: each branch drafts for itself
        c["parent"] = torch.tensor([[-1] + [r.randint(max(0, t - 4), t - 1) for t in range(1, K)] for _ in range(B)], dtype=I32)
    few = torch.randint(0, V, (B, 9), generator=g).to(I32)
    c["tokens"] = torch.gather(few, 1, torch.randint(0, 9, (B, K), generator=g))
    c["tokens"][:, 1::7] = torch.randint(-2, V + 2, (B, len(range(1, K, 7))), generator=g).to(I32)
    c["ids"][:, 1:4] = few[:, :3]                                # with a bias
    c["history"][:, -3:] = few[:, 2:5]                           # in the text, one of them with a bias
    c["params"][:, 2] = 0.05 + 0.1 * torch.rand(B, generator=g)  # (a count too many is seen)
    return c


# how the counts are kept goes by the text's buffer and the number of biases
KEPT = {"16 bits": (90, 5), "parts": (16100, 5), "32 bits": (90, 513)}


@pytest.mark.parametrize("kept", KEPT)
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("B,K,V", [ROWS, (65, 8, 9000), (2, 11, 131072)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_drafts_count_for_their_own_row(B, K, V, tree, kept, dtype):
    say("rows of a workgroup", B, K, V, tree, kept, dtype)
    c = several(B + K, B, K, V, dtype, *KEPT[kept], tree)
    want = expect(c)
    out, b = run(c, F32)
    assert torch.equal(out.cpu(), want) and torch.equal(b.cpu(), ref.best(want))
    # short windows among them: the rows that are there are the same, no other is touched
    r = random.Random(K)
    c["count"] = torch.tensor([r.randint(-1, K + 1) for _ in range(B)], dtype=I32)
    there = torch.arange(K)[None] < c["count"][:, None]
    out, b = run(c, F32)
    assert torch.equal(out.cpu()[there], want[there]) and torch.equal(b.cpu()[there], ref.best(want)[there])
    assert bool((out.cpu()[~there] == 9.0).all()) and bool((b.cpu()[~there] == -7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nothing_to_adjust(dtype):
    """Without parameters and biases the logits come back as they are, whatever is drafted."""
    say("nothing to adjust", dtype)
    c = case(3, *ROWS, 20, dtype, tree=True, params=False)
    out, b = run(c, dtype)
    assert torch.equal(out.cpu(), c["x"]) and torch.equal(b.cpu(), ref.best(c["x"].float()))
