"""The loop of hybrid_loop.py, checked from its record: the cache holds the
accepted tokens' keys and values (equal bits), the pages' counts match the table,
and each window's attention is the plain form's over those tokens."""
import pytest
import torch

from speculative_verify_gdn_amd import gdn, hybrid_loop
from tests import kv_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("kw", [dict(), dict(samples=1, prompt=1, steps=3, N=1), dict(samples=3, prompt=130, N=16, page=32),
                                dict(samples=5, prompt=64, N=5, dtype=torch.float32, D=128, Hq=6)])
def test_loop(kw):
    print("[gpu case] hybrid loop", kw, flush=True)
    cache, rec = hybrid_loop.run(**kw)
    torch.cuda.synchronize()
    samples = cache.lens.numel()
    page, D = cache.page, cache.pool.shape[-1]
    bf16 = cache.pool.dtype == torch.bfloat16
    prompt = [torch.cat([x[i] for x in rec["prompt"]]).cpu() for i in range(2)]          # [tokens][Hkv][D]
    kept = [[p.clone() for p in prompt] for _ in range(samples)]
    for w in rec["windows"]:
        q, o = w["q"].cpu(), w["o"].double().cpu()
        N = q.shape[1]
        assert w["lens"].tolist() == [k[0].shape[0] for k in kept]
        assert w["granted"].tolist() == [N] * samples
        assert bool(torch.isfinite(w["og"]).all())
        parent, node = w["parent"].tolist(), w["node"].tolist()
        for b in range(samples):
            n = kept[b][0].shape[0]
            slots = (n + N + page - 1) // page
            planes = torch.zeros(2, slots * page, cache.pool.shape[2], D, dtype=q.dtype)
            for i, x in enumerate("kv"):
                planes[i, :n], planes[i, n:n + N] = kept[b][i], w[x][b].cpu()
            planes = planes.unflatten(1, (slots, page)).transpose(2, 3).contiguous()
            ro, rl, keys, mean, size = kv_ref.attn(q[b:b + 1], planes[0], planes[1], [n], torch.arange(slots)[None], None,
                                                   [parent[b]])
            to, _ = kv_ref.attn_bounds(ro, rl, keys, mean, size, D, bf16)
            assert float(((o[b:b + 1] - ro).abs() / to).max()) <= 1.0
            path = kv_ref.path(parent[b], node[b]) if node[b] >= 0 else []
            for i, x in enumerate("kv"):
                kept[b][i] = torch.cat([kept[b][i], w[x][b].cpu()[path]])
    table, ref, lens = cache.table.cpu(), cache.ref.tolist(), cache.lens.tolist()
    pool = cache.pool.cpu()
    assert rec["full_lens"].tolist() == [k[0].shape[0] for k in kept]
    count = [0] * len(ref)
    for b in range(samples):
        n = 0 if b in rec["freed"] else kept[b][0].shape[0]
        assert lens[b] == n
        held = (n + page - 1) // page
        assert bool((table[b, held:] == -1).all()) and bool((table[b, :held] >= 0).all())
        for p in table[b, :held].tolist():
            count[p] += 1
        for i in range(2):
            have = pool[i][table[b, :held].long()].transpose(1, 2).flatten(0, 1)[:n]
            assert torch.equal(have, kept[b][i][:n])
    assert count == ref and max(count) <= samples
    used = sum(r > 0 for r in ref)
    assert all(r > 0 for r in ref[:used]), "the pages in use are the lowest"
