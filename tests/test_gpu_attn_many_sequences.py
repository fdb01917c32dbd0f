"""gdn_attn_verify over more sequences than a workgroup has threads (256 in bf16, 512
in fp32) and than it keeps lengths of on chip (512), up to the 4096 of one call."""
import pytest
import torch

from speculative_verify_gdn_amd import gdn
from tests.test_gpu_attn import BF, F32, make, say, trees
from tests.test_gpu_attn_many_rows import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,K,Hq,Hkv,D,page,prefix,own", [
    (257, 2, 4, 2, 64, 16, 0, 70), (511, 1, 2, 1, 128, 16, 0, 200), (513, 3, 3, 1, 64, 32, 96, 40),
    (1100, 1, 4, 2, 256, 16, 64, 33), (1025, 5, 2, 1, 64, 16, 0, 20), (4096, 1, 2, 1, 64, 16, 32, 25)])
def test_many_sequences(dtype, B, K, Hq, Hkv, D, page, prefix, own):
    say("many sequences", dtype, B, K, Hq, Hkv, D, page, prefix, own)
    # every seventh sequence is short of the prefix; lengths of zero among the others
    lens = [max(prefix - 1 - b % 5, 0) if b % 7 == 3 else prefix + b * 37 % own for b in range(B)]
    q, pool, table = make(B, K, Hq, Hkv, D, page, lens, prefix=prefix, dtype=dtype)
    check(q, pool, table, lens, prefix)
    check(q, pool, table, lens, prefix, count=[b * 5 % (K + 1) for b in range(B)], parent=trees(B, K, B))
