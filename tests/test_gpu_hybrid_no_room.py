"""The loop of hybrid_loop.py over a pool too small for all of its windows: a
sequence that got no room keeps the token that its next window starts with."""
import pytest
import torch

from speculative_verify_gdn_amd import gdn, hybrid_loop, synth
from tests.test_gpu_rope import I32, _gpu, say  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_window_without_room():
    say("hybrid loop, one window without room")
    g, gc = torch.Generator(device="cuda").manual_seed(1), torch.Generator().manual_seed(1)
    c = hybrid_loop.Choice(3, 6, 200, 10, 60, g, gc)
    pending, lens = c.next.clone(), c.lens.clone()
    parent = synth.make_tree(3, 6, shape="random").cuda()
    c.step(parent, torch.tensor([6, 0, 6], dtype=I32).cuda())
    assert c.node.tolist()[1] == -1 and min(c.node.tolist()[::2]) >= 0
    assert int(c.next[1]) == int(pending[1]) >= 0 and int(c.lens[1]) == int(lens[1])
    assert bool((c.lens[::2] > lens[::2]).all())


def test_a_pool_too_small(monkeypatch):
    say("hybrid loop, a pool too small")

    class Small(hybrid_loop.Cache):
        """Room for the prompt's four pages and one window each for two of the three sequences."""

        def __init__(self, samples, slots, n_pages, *rest):
            super().__init__(samples, slots, 6, *rest)

    monkeypatch.setattr(hybrid_loop, "Cache", Small)
    _, rec = hybrid_loop.run(samples=3, prompt=64, steps=6, vocab=500)
    torch.cuda.synchronize()
    certain, without, lens = None, 0, None
    for w in rec["windows"]:
        w = {k: w[k].cpu() for k in ("granted", "tokens", "next", "node", "text_lens", "text")}
        if certain is not None:
            assert torch.equal(w["tokens"][:, 0], certain)
        for b in range(3):
            assert bool((w["text"][b, :int(w["text_lens"][b])] >= 0).all())
            if int(w["granted"][b]) == 0:
                without += 1
                assert int(w["node"][b]) == -1 and int(w["next"][b]) == int(w["tokens"][b, 0])
            else:
                assert int(w["node"][b]) >= 0
        assert int(w["next"].min()) >= 0
        certain = w["next"]
    assert without > 0
    text, n = rec["text"].cpu(), rec["text_lens"].tolist()
    assert all(bool((text[b, :n[b]] >= 0).all()) for b in range(3))
