"""gdn_attn_verify where scores are far from zero: the weights depend on the
differences of a row's scores alone, however large the scores are.

The scores here are exact in float (products of powers of two and small whole
numbers, one non-zero column), so the weights of tied keys are exactly equal and
those of the others exactly zero, and the bound counts the sums and the output's
rounding only (kv_ref.attn_bounds with a score size of 0)."""
import pytest
import torch

from speculative_verify_gdn_amd import gdn
from tests import kv_ref
from tests.test_gpu_attn import BF, F32, dev, make, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.load()
    yield
    torch.cuda.synchronize()


def put(pool, table, b, page, pos, column):
    """Sets the keys at positions `pos` of sequence b to (column, 0, 0, ..)."""
    for n, c in zip(pos, column):
        pool[0, table[b][n // page], :, n % page] = 0
        pool[0, table[b][n // page], :, n % page, 0] = c


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("q0,unit,n", [
    (2.0 ** 15, 2.0 ** 20, 600),       # scores of 2^32 and more, steps of 2^32
    (2.0 ** 15, -2.0 ** 20, 600),
    (2.0 ** 60, 2.0 ** 50, 70),        # 2^107 and more
    (2.0 ** 60, -2.0 ** 62, 300),      # down to -2^124: far below -1e37
    (2.0 ** 10, 2.0 ** 12, 300),       # references on both sides of where the form of the exponents changes
])
@pytest.mark.parametrize("prefix", [0, 64])
def test_scores_far_from_zero(dtype, D, q0, unit, n, prefix):
    say("far", dtype, D, q0, unit, n, prefix)
    K, Hq, Hkv, page = 3, 4, 2, 16
    lens = [n, max(prefix, 40)]
    q, pool, table = make(21, K, Hq, Hkv, D, page, lens, prefix=prefix, dtype=dtype)
    q.zero_()
    q[..., 0] = q0
    for b, length in enumerate(lens):
        pos = range(length + K)
        put(pool, table, b, page, pos, [unit * (1 + (7 * i + i // 5) % 4) for i in pos])
    dq, dp, dl, dt = q.cuda(), pool.cuda(), dev(lens), dev(table)
    o, lse = torch.zeros_like(dq), torch.zeros(2, K, Hq, device="cuda")
    gdn.attn_verify(dq, dp[0], dp[1], dl, dt, o, prefix_len=prefix, lse=lse, scale=0.125,
                    workspace=gdn.attn_workspace(dq, dp[0], dt, prefix))
    torch.cuda.synchronize()
    ro, rl, keys, mean, size = kv_ref.attn(q, pool[0], pool[1], lens, torch.tensor(table), scale=0.125)
    to, tl = kv_ref.attn_bounds(ro, rl, keys, mean, torch.zeros_like(size), D, dtype == BF)
    err = (o.double().cpu() - ro).abs() / to
    assert bool(torch.isfinite(o).all()) and float(err.max()) <= 1.0
    assert float(((lse.double().cpu() - rl).abs() / tl).max()) <= 1.0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_far_row_beside_ordinary_ones(dtype):
    """One head's rows are far, the others ordinary: each is what it is alone."""
    say("far beside ordinary", dtype)
    K, Hq, Hkv, D, page, n = 4, 8, 1, 64, 16, 333
    q, pool, table = make(22, K, Hq, Hkv, D, page, [n], dtype=dtype)
    dp, dl, dt = pool.cuda(), dev([n]), dev(table)

    def run(x):
        dq, o = x.cuda(), torch.zeros(x.shape, dtype=dtype, device="cuda")
        gdn.attn_verify(dq, dp[0], dp[1], dl, dt, o, workspace=gdn.attn_workspace(dq, dp[0], dt))
        return o.cpu()

    plain = run(q)
    far = q.clone()
    far[:, :, 3] *= 2.0 ** 40
    mixed = run(far)
    others = [h for h in range(Hq) if h != 3]
    assert torch.equal(mixed[:, :, others], plain[:, :, others])
    assert bool(torch.isfinite(mixed).all())
    # the far rows are the value of their best key (a key with the greatest score; the gaps are far above 2^30)
    keys = torch.cat([pool[0, table[0][s], 0] for s in range((n + K + page - 1) // page)])[:n + K].double()
    values = torch.cat([pool[1, table[0][s], 0] for s in range((n + K + page - 1) // page)])[:n + K]
    for t in range(K):
        best = int((keys[:n + t + 1] @ far[0, t, 3].double()).argmax())
        assert torch.equal(mixed[0, t, 3], values[best])
