"""The loop of hybrid_loop.py with a vocabulary: norms and rotations on the way
into the cache, logits that choose the accepted node.  The cache and the attention
are checked as without one, and the choice against the plain forms."""
import pytest
import torch

from speculative_verify_gdn_amd import gdn, hybrid_loop
from tests import test_gpu_hybrid_loop as plain
from tests import window_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.load()
    yield
    torch.cuda.synchronize()


CASES = [dict(vocab=1000), dict(vocab=503, samples=1, prompt=1, steps=3, N=1), dict(vocab=3000, samples=3, prompt=130, N=16, page=32),
         dict(vocab=777, samples=5, prompt=64, N=5, dtype=torch.float32, D=128, Hq=6)]


@pytest.mark.parametrize("kw", CASES)
def test_cache_and_attention(kw):
    plain.test_loop(kw)


@pytest.mark.parametrize("kw", CASES)
def test_the_choice(kw):
    print("[gpu case] hybrid loop's choice", kw, flush=True)
    _, rec = hybrid_loop.run(**kw)
    torch.cuda.synchronize()
    start, params = rec["text_start"].cpu(), rec["params"].cpu()
    accepted, certain = [], None
    for w in rec["windows"]:
        c = {k: w[k].cpu() for k in ("logits", "text", "text_lens", "tokens", "parent", "best", "next", "node")}
        if certain is not None:
            assert torch.equal(c["tokens"][:, 0], certain)   # a window starts with the token the one before it ended on
        f32 = ref.logits(c["logits"], c["text"], c["text_lens"], start, c["tokens"], c["parent"].tolist(), params)[1]
        assert torch.equal(c["best"], ref.best(f32))
        node, nxt, text, lens = ref.accept(c["best"].tolist(), c["tokens"].tolist(), c["parent"].tolist(), None, None,
                                           c["text"].tolist(), c["text_lens"].tolist())
        assert c["node"].tolist() == node and c["next"].tolist() == nxt
        certain = c["next"]
        accepted += node
    assert rec["text"].cpu().tolist() == text and rec["text_lens"].tolist() == lens
    assert min(accepted) >= 0
    if kw.get("N", 8) > 1:
        assert max(accepted) > 0
