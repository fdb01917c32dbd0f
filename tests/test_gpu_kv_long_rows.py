"""kv_rollback_tree and kv_reserve where a table row is longer than what the
kernels keep on chip (2048 slots), and at that border, against the Python loops."""
import pytest
import torch

from speculative_verify_gdn_amd import gdn
from tests import kv_ref
from tests.test_gpu_kv import dev, make_pool, say, state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("P", [2047, 2048, 2049, 4100])
@pytest.mark.parametrize("planes", [1, 200])
@pytest.mark.parametrize("inplace", [False, True])
def test_rollback(P, planes, inplace):
    say("rollback long rows", P, planes, inplace)
    B, N, Hkv, page, D, n_pages = 3, 9, 1, 16, 64, 60
    lens, table, ref = state(5, B, P, n_pages, page, 150)
    g = torch.Generator().manual_seed(6)
    pool = make_pool(g, planes, n_pages, Hkv, page, D, torch.bfloat16)
    # one sequence ends at the end of its row: its pages moved to the last slots, the others stay in front
    held = sum(x >= 0 for x in table[1])
    table[1] = [-1] * (P - held) + table[1][:held]
    lens[1] = P * page - 4
    parent = [[-1, 0, 0, 1, 2, 3, 3, 5, 6]] * B
    node, count = [8, 4, 6], [9, 9, 7]
    d = [dev(x) for x in (node, parent, lens, table, ref)]
    dp = pool.cuda()
    out = d[2] if inplace else dev([0] * B)
    gdn.kv_rollback_tree(d[0], d[1], d[2], d[3], d[4], dp, out, count=dev(count))
    want = kv_ref.rollback(node, parent, lens, table, ref, pool, N, count)
    assert out.tolist() == want
    assert d[3].tolist() == table and d[4].tolist() == ref
    assert torch.equal(dp.cpu(), pool)


@pytest.mark.parametrize("B,n_pages", [(1024, 4096), (1025, 4096), (1024, 4097), (1, 4096), (300, 260)])
def test_reserve_at_the_border(B, n_pages):
    """Both kernels at the sizes where one takes over from the other; windows of many slots."""
    say("reserve border", B, n_pages)
    P, page = 12, 16
    lens, table, ref = state(7, B, P, n_pages, page, 40)
    add = [(37 * b) % 120 for b in range(B)]
    d = [dev(x) for x in (lens, add, table, ref)]
    granted = dev([7] * B)
    gdn.kv_reserve(d[0], d[1], d[2], d[3], page, granted)
    assert kv_ref.reserve(lens, add, table, ref, page) == granted.tolist()
    assert d[2].tolist() == table and d[3].tolist() == ref
