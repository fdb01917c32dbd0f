"""kv_fork and kv_reserve over pools of several scan steps (4096 pages each) and with
several forks a thread (above 1024), against the Python loops: free pages on both
sides of a step's border, in the last step alone, and too few of them."""
import random

import pytest
import torch

from speculative_verify_gdn_amd import gdn
from tests import kv_ref
from tests.test_gpu_kv import dev, make_pool, say

pytestmark = pytest.mark.gpu
HKV, PAGE, D, P = 1, 16, 64, 3


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.load()
    yield
    torch.cuda.synchronize()


def cache(n, n_pages, free):
    """n + 3 rows: two prompts of 37 and 32 tokens, an empty one, rows to fork into; all pages outside `free` in use."""
    ref = [0 if p in free else 1 for p in range(n_pages)]
    table = [[-1] * P for _ in range(n + 3)]
    lens = [37, 32] + [0] * (n + 1)
    used = [p for p in range(n_pages) if ref[p]]
    random.Random(n).shuffle(used)
    table[0], table[1][:2] = used[:3], used[3:5]
    return lens, table, ref


def spread(lo, hi, k, seed):
    return set(random.Random(seed).sample(range(lo, hi), k))


@pytest.mark.parametrize("n,n_pages,free", [
    (1025, 4096, spread(0, 4096, 1100, 1)),
    (1025, 9000, spread(3000, 5200, 1500, 2)),                # across the first border
    (4096, 12000, spread(0, 4096, 700, 3) | spread(8192, 12000, 2500, 4)),
    (4096, 4097, {4096}),                                     # one page, in the second step
    (2000, 8200, spread(0, 8192, 800, 5) | set(range(8192, 8200))),   # runs out in the third step
    (64, 8193, {4095, 4096, 8191, 8192}),                     # a fork a thread, runs out
    (30, 5000, set()),
])
def test_fork(n, n_pages, free):
    say("fork large", n, n_pages, len(free))
    lens, table, ref = cache(n, n_pages, free)
    r = random.Random(n + n_pages)
    src = [r.choice([0, 0, 0, 1, 2, -1]) for _ in range(n)]
    dst = list(range(3, n + 3))
    r.shuffle(dst)
    pool = make_pool(torch.Generator().manual_seed(n), 2, n_pages, HKV, PAGE, D, torch.bfloat16)
    dp, dl, dt, dr = pool.cuda(), dev(lens), dev(table), dev(ref)
    granted = dev([7] * n)
    gdn.kv_fork(dev(src), dev(dst), dl, dt, dr, dp, granted)
    want = kv_ref.fork(src, dst, lens, table, ref, pool)
    assert granted.tolist() == want
    assert dl.tolist() == lens and dt.tolist() == table and dr.tolist() == ref
    assert torch.equal(dp.cpu(), pool)


@pytest.mark.parametrize("B,n_pages,free", [
    (1500, 9000, spread(3000, 5200, 1500, 2)), (3000, 12000, spread(0, 4096, 700, 3) | spread(8192, 12000, 2500, 4)),
    (9, 70000, spread(60000, 70000, 40, 6)), (2000, 8200, spread(0, 8192, 800, 5) | set(range(8192, 8200)))])
def test_reserve(B, n_pages, free):
    say("reserve large", B, n_pages, len(free))
    lens, table, ref = cache(B - 3, n_pages, free)
    r = random.Random(B)
    add = [r.choice([0, 1, 16, 17, 48]) for _ in range(B)]
    dl, dt, dr, granted = dev(lens), dev(table), dev(ref), dev([7] * B)
    gdn.kv_reserve(dl, dev(add), dt, dr, PAGE, granted)
    assert kv_ref.reserve(lens, add, table, ref, PAGE) == granted.tolist()
    assert dt.tolist() == table and dr.tolist() == ref
