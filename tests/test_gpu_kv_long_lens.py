"""The cache calls where a length is at the end of its 31 bits, far behind the
table's slots: nothing is moved, stored, taken or given back, and the length that
kv_rollback_tree leaves does not wrap."""
import pytest
import torch

from speculative_verify_gdn_amd import gdn
from tests.test_gpu_kv import dev, make_pool, say

pytestmark = pytest.mark.gpu
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("planes", [2, 200])       # one kernel, and two
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("P", [4, 2100])           # the row kept on chip, and not
def test_rollback(planes, inplace, P):
    say("rollback at the last length", planes, inplace, P)
    g = torch.Generator().manual_seed(1)
    lens = [TOP, TOP - 2, TOP - 20, 20]
    n_pages, page, N = 12, 16, 9
    table = [[3 * b, 3 * b + 1, 3 * b + 2] + [-1] * (P - 3) for b in range(4)]
    ref = [1] * n_pages
    pool = make_pool(g, planes, n_pages, 1, page, 64, torch.bfloat16)
    d = [dev(x) for x in (lens, table, ref)]
    dp = pool.cuda()
    out = d[0] if inplace else dev([5] * 4)
    gdn.kv_rollback_tree(dev([8, 8, 8, 8]), None, d[0], d[1], d[2], dp, out, N=N)
    assert out.tolist() == [TOP, TOP, TOP - 11, 29]
    table[3][2], ref[11] = -1, 0                    # 29 tokens: two pages
    assert d[1].tolist() == table and d[2].tolist() == ref
    assert torch.equal(dp.cpu(), pool)


def test_other_calls():
    say("other calls at the last length")
    g = torch.Generator().manual_seed(2)
    B, P, n_pages, page, K = 2, 3, 8, 16, 5
    table, ref = [[0, 1, 2], [3, 4, -1]], [1] * 5 + [0] * 3
    pool = make_pool(g, 2, n_pages, 2, page, 64, torch.bfloat16)
    dl, dt, dr, dp = dev([TOP, TOP - 3]), dev(table), dev(ref), pool.cuda()
    granted = dev([7, 7])
    gdn.kv_reserve(dl, dev([1, TOP]), dt, dr, page, granted)
    assert granted.tolist() == [0, 0]
    k = torch.ones(B, K, 2, 64, dtype=torch.bfloat16, device="cuda")
    gdn.kv_append(k, k, dp[0], dp[1], dl, dt)
    gdn.kv_fork(dev([0]), dev([1]), dl, dt, dr, dp, granted[:1])
    assert granted.tolist() == [0, 0]
    assert dt.tolist() == table and dr.tolist() == ref and dl.tolist() == [TOP, TOP - 3]
    assert torch.equal(dp.cpu(), pool)
