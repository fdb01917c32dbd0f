"""gdn_attn_verify where scores are -infinity (keys that a caller pushed there): such
a key has no weight, and a row all of whose scores are -infinity is the formula's
0 / 0, NaN with lse = -inf.  Only a row that sees no key has o = 0."""
import math

import pytest
import torch

from speculative_verify_gdn_amd import gdn
from tests import kv_ref
from tests.test_gpu_attn import BF, F32, dev, make, say, trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.load()
    yield
    torch.cuda.synchronize()


def push(pool, table, b, page, h, positions):
    """The keys of head h at `positions` of sequence b: -inf in column 0, so -inf is every score of a q above 0 there."""
    for n in positions:
        pool[0, table[b][n // page], h, n % page, 0] = -math.inf


def check(q, pool, table, lens, prefix=0, count=None, parent=None):
    B, K, Hq, D = q.shape
    dq, dp, dt = q.cuda(), pool.cuda(), dev(table)
    o, lse = torch.full_like(dq, 7.0), torch.full((B, K, Hq), 7.0, device="cuda")
    work = gdn.attn_workspace(dq, dp[0], dt, prefix)
    work.fill_(0xFF)
    gdn.attn_verify(dq, dp[0], dp[1], dev(lens), dt, o, prefix_len=prefix, count=None if count is None else dev(count),
                    parent=None if parent is None else dev(parent), lse=lse, workspace=work)
    torch.cuda.synchronize()
    # the bound's score size over finite keys: a key without weight adds no rounding
    tame = pool.clone()
    tame[0][torch.isinf(tame[0])] = 0
    size = kv_ref.attn(q, tame[0], tame[1], lens, torch.tensor(table), count, parent)[4]
    ro, rl, keys, mean, _ = kv_ref.attn(q, pool[0], pool[1], lens, torch.tensor(table), count, parent)
    to, tl = kv_ref.attn_bounds(ro, rl, keys, mean, size, D, q.dtype == BF)
    live = torch.ones(B, K, dtype=torch.bool) if count is None else torch.arange(K)[None] < torch.tensor(count)[:, None]
    go, gl, live = o.double().cpu(), lse.double().cpu(), live[..., None].expand(B, K, Hq)
    nan, none = torch.isnan(ro[..., 0]) & live, (keys == 0) & live
    assert bool(torch.isnan(go[nan]).all()) and bool((gl[nan] == -math.inf).all())
    assert bool((go[none] == 0).all()) and bool((gl[none] == -math.inf).all())
    some = live & ~nan & ~none
    assert bool(torch.isfinite(go[some]).all()) and bool(((go - ro).abs() <= to)[some].all())
    assert bool(((gl - rl).abs() <= tl)[some].all())
    return int(nan.sum()), int(none.sum()), int(some.sum())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,K,Hq,page,n,prefix", [
    (1, 1, 4, 16, 40, 0), (2, 5, 8, 16, 900, 0), (3, 9, 12, 64, 70, 256), (4, 1, 8, 32, 200, 1024), (1, 64, 4, 16, 33, 0),
    (2, 40, 64, 16, 150, 64)])
def test_scores_of_minus_infinity(dtype, D, B, K, Hq, page, n, prefix):
    say("minus infinity", dtype, D, B, K, Hq, page, n, prefix)
    Hkv = 4
    lens = [prefix + n - b for b in range(B)]
    q, pool, table = make(D + K, K, Hq, Hkv, D, page, lens, prefix=prefix, dtype=dtype)
    q[..., 0] = q[..., 0].abs() + 0.5
    # head 0: every key; 1: the committed ones; 2: the first half of them; 3: all but a late committed one
    for b, length in enumerate(lens):
        push(pool, table, b, page, 0, range(length + K))
        push(pool, table, b, page, 1, range(length))
        push(pool, table, b, page, 2, range(length // 2))
        push(pool, table, b, page, 3, [i for i in range(length + K) if i != length - 3])
    nan, none, some = check(q, pool, table, lens, prefix)
    assert nan == B * K * Hq // Hkv and none == 0 and some == 3 * nan
    # trees: rows see other nodes, and in head 1 none but their path's
    for b, length in enumerate(lens):
        push(pool, table, b, page, 1, range(length + K // 2))
    count = [max(K - b, 1) for b in range(B)]
    nan, none, _ = check(q, pool, table, lens, prefix, count=count, parent=trees(B, K, D))
    assert nan > 0 and none == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K,page,prefix", [(1, 16, 0), (6, 16, 48), (33, 32, 64)])
def test_beside_missing_pages(dtype, K, page, prefix):
    """Pages that are missing and keys without weight: which of the two a row has decides between 0 and NaN."""
    say("minus infinity, missing pages", dtype, K, page, prefix)
    Hq, Hkv, D, n = 4, 2, 128, 200
    lens = [prefix + n] * 4
    q, pool, table = make(K, K, Hq, Hkv, D, page, lens, prefix=prefix, dtype=dtype)
    q[..., 0] = q[..., 0].abs() + 0.5
    for b, length in enumerate(lens):
        push(pool, table, b, page, 0, range(length + K))
    P, own = len(table[0]), prefix // page
    table[1] = [-1] * P                                     # sees nothing
    if prefix:
        for row in table:
            row[:own] = [-1] * own                          # (nobody holds the prefix)
    table[2] = table[2][:own] + [-1] * (P - own - 1) + table[2][-1:]  # only its last page
    nan, none, some = check(q, pool, table, lens, prefix)
    assert none >= K * Hq and nan > 0 and some > 0
    check(q, pool, table, lens, prefix, parent=trees(4, K, 1))
    check(q, pool, table, lens, prefix, count=[K, K, max(K - 1, 1), 1])
