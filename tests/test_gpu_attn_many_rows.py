"""gdn_attn_verify with many query rows a key/value head: the numbers of row tiles
at which they stop having a workgroup each, on both sides, within the counted
bound of the 64-bit plain form; and the same bits from another stream, ordered
after what the first one wrote."""
import pytest
import torch

from speculative_verify_gdn_amd import gdn
from tests import kv_ref
from tests.test_gpu_attn import BF, F32, dev, make, say, trees

pytestmark = pytest.mark.gpu
MARK = 7.0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.load()
    yield
    torch.cuda.synchronize()


def check(q, pool, table, lens, prefix=0, count=None, parent=None):
    B, K, Hq, D = q.shape
    dq, dp, dl, dt = q.cuda(), pool.cuda(), dev(lens), dev(table)
    o, lse = torch.full_like(dq, MARK), torch.full((B, K, Hq), MARK, device="cuda")
    work = gdn.attn_workspace(dq, dp[0], dt, prefix)
    work.fill_(0xFF)                                        # (NaN: what nobody wrote shows)
    kw = dict(prefix_len=prefix, count=None if count is None else dev(count), parent=None if parent is None else dev(parent),
              workspace=work)
    gdn.attn_verify(dq, dp[0], dp[1], dl, dt, o, lse=lse, **kw)
    again = torch.full_like(o, MARK)
    work.fill_(0xFF)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    gdn.attn_verify(dq, dp[0], dp[1], dl, dt, again, stream=side, **kw)
    torch.cuda.synchronize()
    assert torch.equal(o, again)
    ro, rl, keys, mean, size = kv_ref.attn(q, pool[0], pool[1], lens, torch.tensor(table), count, parent)
    to, tl = kv_ref.attn_bounds(ro, rl, keys, mean, size, D, q.dtype == BF)
    live = torch.ones(B, K, dtype=torch.bool) if count is None else torch.arange(K)[None] < torch.tensor(count)[:, None]
    go, gl = o.double().cpu(), lse.double().cpu()
    assert bool((go[~live] == MARK).all()) and bool((gl[~live] == MARK).all())
    assert bool(torch.isfinite(go[live]).all())
    assert float(((go - ro).abs() / to)[live].max()) <= 1.0
    assert float(((gl - rl).abs() / tl)[live].max()) <= 1.0


@pytest.mark.parametrize("dtype,D,K,Hq,Hkv,page,lens,prefix", [
    (BF, 256, 64, 1024, 1, 16, [50], 0),          # 1024 row tiles of 64 rows, 512 workgroups
    (BF, 256, 64, 1024, 1, 16, [33, 40], 32),
    (BF, 256, 33, 1024, 1, 32, [70], 0),          # 528
    (BF, 256, 32, 1024, 1, 32, [70, 5], 0),       # 512: a workgroup each
    (BF, 128, 64, 1024, 1, 16, [40], 0),          # 512 of 128 rows
    (F32, 64, 33, 1024, 1, 16, [50], 0),          # 264 of 128 rows, 256 workgroups
    (F32, 64, 64, 1024, 1, 16, [16, 3], 16),
    (F32, 128, 33, 993, 1, 16, [300], 0),         # 257
    (F32, 64, 32, 1024, 1, 16, [90], 0),          # 256
    (F32, 256, 64, 1024, 1, 64, [128, 65], 64),
])
def test_more_row_tiles_than_workgroups(dtype, D, K, Hq, Hkv, page, lens, prefix):
    say("many rows", dtype, D, K, Hq, Hkv, page, lens, prefix)
    q, pool, table = make(K + D, K, Hq, Hkv, D, page, lens, prefix=prefix, dtype=dtype)
    check(q, pool, table, lens, prefix)
    if len(lens) > 1:
        check(q, pool, table, lens, prefix, count=[K, K // 2], parent=trees(len(lens), K, 5))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,K,Hq,Hkv,page,prefix,own", [
    (64, 40, 8, 2, 16, 0, [700, 0, 33]), (128, 64, 12, 4, 32, 256, [3, 90]), (256, 5, 24, 4, 64, 512, [1, 200, 64])])
def test_another_stream_gives_the_same_bits(dtype, D, K, Hq, Hkv, page, prefix, own):
    say("another stream", dtype, D, K, Hq, Hkv, page, prefix, own)
    lens = [prefix + n for n in own]
    q, pool, table = make(D, K, Hq, Hkv, D, page, lens, prefix=prefix, dtype=dtype)
    check(q, pool, table, lens, prefix)
    check(q, pool, table, lens, prefix, count=[max(K - 3 * b, 0) for b in range(len(lens))])
