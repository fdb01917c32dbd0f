"""A speculative decoding loop of a hybrid model's two kinds of layer, one of
each, as a serving program runs it on these calls:

  prompt   in windows of up to 64 tokens: pages reserved, keys and values
           appended, the window attended (kv_reserve, kv_append, attn_verify),
           the GDN layer's conv and recurrence (conv_step, verify)
  fork     the prompt's sequence forked into the samples: full pages shared, the
           partial last one copied (kv_fork); the GDN state copied
  steps    a draft tree a sample: pages, append, attention of the tree over the
           cache with the shared prompt read once (attn_verify, prefix_len), the
           GDN layer's tree step (verify_tree_step), then both layers cut back to
           the accepted node (kv_rollback_tree; the next verify_tree_step)
  end      half of the samples freed, the pool made dense (kv_free, kv_compact)

The projections, the drafts and the choice of the accepted node are drawn at
random (they are the model's business); what runs here is the cache, the
attention and the recurrence.  With a vocabulary (run(vocab=...)) the loop is
closed: queries and keys are normed and turned to their positions on the way
into the cache (kv_append_rope), the nodes' logits, drawn at random, adjusted for
the tokens seen so far (logits_adjust), and the accepted node is the deepest one
that they confirm (accept_tree).  `python -m speculative_verify_gdn_amd.hybrid_loop`
runs both and prints what they did.
"""
from __future__ import annotations

import torch

from . import gdn, synth

I32 = torch.int32


class Front:
    """What queries and keys pass on their way in: the norms' weights, and the frequencies of the part of a head that
    turns (a quarter), scaled for contexts of 8 x 4096 tokens."""

    def __init__(self, D, g, device="cuda"):
        self.wq, self.wk = (1.0 + 0.1 * torch.randn(D, generator=g, device=device) for _ in range(2))
        self.freqs, self.mscale = gdn.rope_freqs(D // 4, 1e6, "yarn", 8.0, original=4096, device=device)

    def pass_in(self, cache, row, Hq, rows, parent, granted):
        """The stacked projection rows [B][K][(Hq + 2 Hkv) D] of a window: keys and values into the cache; the queries."""
        Hkv, D = cache.pool.shape[2], cache.pool.shape[-1]
        q, k, v = (x.unflatten(-1, (-1, D)) for x in row.split((Hq * D, Hkv * D, Hkv * D), -1))
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        gdn.kv_append_rope(k, v, cache.pool[0], cache.pool[1], cache.lens[:rows], cache.table[:rows], self.freqs, q=q, q_out=out,
                           wq=self.wq, wk=self.wk, parent=parent, count=granted, mscale=self.mscale)
        return out


class Cache:
    """The paged cache of one attention layer: pool [2][n_pages][Hkv][page][D], a table row and a length for each
    sequence, and the users of each page."""

    def __init__(self, rows, slots, n_pages, Hkv, page, D, dtype, device="cuda"):
        self.pool = torch.zeros(2, n_pages, Hkv, page, D, dtype=dtype, device=device)
        self.table = torch.full((rows, slots), -1, dtype=I32, device=device)
        self.lens = torch.zeros(rows, dtype=I32, device=device)
        self.ref = torch.zeros(n_pages, dtype=I32, device=device)
        self.page = page

    def window(self, q, k, v, o, rows, parent=None, prefix_len=0, workspace=None, pass_in=None):
        """Room for a window of the first `rows` sequences, its keys and values in place, its attention in o.  pass_in:
        puts the keys and values there itself and returns the queries (q: their shape)."""
        K = q.shape[1]
        add = torch.full((rows,), K, dtype=I32, device=q.device)
        granted = torch.empty_like(add)
        lens, table = self.lens[:rows], self.table[:rows]
        gdn.kv_reserve(lens, add, table, self.ref, self.page, granted)
        if pass_in is not None:
            q = pass_in(granted)
        else:
            gdn.kv_append(k, v, self.pool[0], self.pool[1], lens, table, count=granted)
        if workspace is None:
            workspace = gdn.attn_workspace(q, self.pool[0], table, prefix_len)
        gdn.attn_verify(q, self.pool[0], self.pool[1], lens, table, o, prefix_len=prefix_len, count=granted,
                        parent=parent, workspace=workspace)
        return granted

    def accept(self, node, parent, granted, rows, N=None):
        """The first `rows` sequences keep the path to node of their window (parent None: a chain of N)."""
        lens = self.lens[:rows]
        gdn.kv_rollback_tree(node, parent, lens, self.table[:rows], self.ref, self.pool, lens, count=granted, N=N)

    def compact(self):
        work = gdn.kv_compact_workspace(self.ref)
        table, ref = torch.empty_like(self.table), torch.empty_like(self.ref)
        gdn.kv_compact(self.table, self.ref, self.pool, table, ref, work)
        self.table, self.ref = table, ref


class Choice:
    """The other end: logits of every node, the tokens they confirm, and the text that grows by them."""

    def __init__(self, samples, N, vocab, prompt, room, g, gc, device="cuda"):
        self.vocab, self.g, self.gc = vocab, g, gc
        self.history = torch.randint(0, vocab, (1, prompt + room), generator=g, device=device, dtype=I32).repeat(samples, 1)
        self.lens = torch.full((samples,), prompt, dtype=I32, device=device)
        self.start = self.lens.clone()
        self.params = torch.tensor([1.1, 0.2, 0.1, 0.8], device=device).repeat(samples, 1)
        self.best = torch.empty(samples, N, dtype=I32, device=device)
        self.node, self.next = (torch.empty(samples, dtype=I32, device=device) for _ in range(2))
        self.next.random_(0, vocab, generator=g)
        self.workspace = None

    def step(self, parent, granted):
        """Draft tokens for the nodes of `parent` (the root's is the last step's next one), adjusted logits, the accepted
        node; returns what went in."""
        samples, N = parent.shape
        logits = torch.randn(samples, N, self.vocab, generator=self.g, device=parent.device) * 2
        # the drafter is right about the plain best of its parent three times of four
        guess = torch.gather(logits.argmax(-1), 1, parent.long().clamp(min=0)).to(I32)
        other = torch.randint(0, self.vocab, (samples, N), generator=self.g, device=parent.device, dtype=I32)
        tokens = torch.where(torch.rand(samples, N, generator=self.g, device=parent.device) < 0.75, guess, other)
        tokens[:, 0] = self.next
        if self.workspace is None:
            self.workspace = gdn.logits_workspace(logits)
        before = dict(logits=logits, tokens=tokens, text=self.history.clone(), text_lens=self.lens.clone())
        gdn.logits_adjust(logits, best=self.best, history=self.history, history_lens=self.lens, history_start=self.start,
                          tokens=tokens, parent=parent, count=granted, params=self.params, workspace=self.workspace)
        # (a sequence that got no room has no node to accept: its next token stays the one that it began with)
        gdn.accept_tree(self.best, tokens, self.node, self.next, parent=parent, count=granted, root=tokens[:, 0].contiguous(),
                        history=self.history, lens=self.lens, lens_out=self.lens)
        return dict(before, best=self.best.clone(), next=self.next.clone())


def run(samples=4, prompt=200, steps=5, N=8, Hq=8, Hkv=2, D=64, page=16, dtype=torch.bfloat16, seed=0, vocab=0):
    """The loop; returns the cache and a record of what went into it (for a check against plain attention)."""
    wl = synth.small("verify16", B=samples, T=N, Hk=2, Hv=4, dk=64, dv=64)
    g = torch.Generator(device="cuda").manual_seed(seed)
    gc = torch.Generator().manual_seed(seed + 1)

    def rand(*shape, t=dtype):
        return torch.randn(*shape, generator=g, device="cuda").to(t)

    slots = (prompt + steps * N + page - 1) // page + 1
    n_pages = prompt // page + samples * ((steps + 1) * N // page + 2)
    cache = Cache(samples, slots, n_pages, Hkv, page, D, dtype)
    w, dt_bias, A_log = rand(wl.C, wl.W, t=torch.float32) * 0.5, rand(wl.Hv, t=torch.float32), rand(wl.Hv, t=torch.float32)
    io = torch.bfloat16
    front = Front(D, g) if vocab else None
    choice = Choice(samples, N, vocab, prompt, (steps + 1) * N, g, gc) if vocab else None

    def turned(row, lens, parent):
        """The queries and keys of projection rows as they come out of the front, and the values (for the record)."""
        q, k, v = (x.unflatten(-1, (-1, D)) for x in row.split((Hq * D, Hkv * D, Hkv * D), -1))
        qt, kt = (torch.empty(x.shape, dtype=dtype, device="cuda") for x in (q, k))
        gdn.qk_norm_rope(q, k, front.wq, front.wk, front.freqs, qt, kt, lens=lens, parent=parent, mscale=front.mscale)
        return qt, kt, v

    # the prompt, in row 0
    hist = torch.zeros(1, wl.W - 1, wl.C, dtype=io, device="cuda")
    S = torch.zeros(1, wl.Hv, wl.dv, wl.dk, device="cuda")
    kept = []                      # keys and values of the tokens that row 0 committed
    for at in range(0, prompt, 64):
        K = min(64, prompt - at)
        into = None
        if front:
            row = rand(1, K, (Hq + 2 * Hkv) * D)
            q, k, v = turned(row, cache.lens[:1], None)
            into = lambda granted: front.pass_in(cache, row, Hq, 1, None, granted)
        else:
            q, k, v = rand(1, K, Hq, D), rand(1, K, Hkv, D), rand(1, K, Hkv, D)
        granted = cache.window(q, k, v, torch.empty_like(q), rows=1, pass_in=into)
        cache.accept(torch.full((1,), K - 1, dtype=I32, device="cuda"), None, granted, rows=1, N=K)
        x, y = rand(1, K, wl.C, t=io), torch.empty(1, K, wl.C, dtype=io, device="cuda")
        win = torch.empty(1, wl.W - 1 + K, wl.C, dtype=io, device="cuda")
        S_out, o = torch.empty_like(S), torch.empty(1, K, wl.Hv, wl.dv, dtype=io, device="cuda")
        H = torch.empty(1, K - 1, wl.Hv, wl.dv, wl.dk, device="cuda") if K > 1 else None
        gdn.conv_step(x, w, hist, y, win)
        gdn.verify(y, rand(1, K, wl.Hv, t=io), rand(1, K, wl.Hv, t=io), dt_bias, A_log, S, S_out, H, o, wl.Hk)
        S = S_out
        kept.append((k[0], v[0]))

    # one sequence becomes `samples`
    if samples > 1:
        dst = torch.arange(1, samples, dtype=I32, device="cuda")
        granted = torch.empty_like(dst)
        gdn.kv_fork(torch.zeros_like(dst), dst, cache.lens, cache.table, cache.ref, cache.pool, granted)
    prefix = prompt // page * page

    # tree steps; the GDN layer alternates two sets of buffers, its rollback is the next step's first part
    sets = [dict(S=torch.empty(samples, wl.Hv, wl.dv, wl.dk, device="cuda"),
                 H=torch.empty(samples, N, wl.Hv, wl.dv, wl.dk, device="cuda"),
                 hist=torch.empty(samples, wl.W - 1, wl.C, dtype=io, device="cuda")) for _ in range(2)]
    S_prev, hist_prev, prev = S.expand(samples, -1, -1, -1).contiguous(), hist.expand(samples, -1, -1).contiguous(), None
    workspace, windows = None, []
    for i in range(steps):
        parent = synth.make_tree(samples, N, seed=seed + i, shape="random").cuda()
        into, more = None, {}
        if front:
            row = rand(samples, N, (Hq + 2 * Hkv) * D)
            q, k, v = turned(row, cache.lens, parent)
            into = lambda granted: front.pass_in(cache, row, Hq, samples, parent, granted)
        else:
            node = torch.randint(-1, N, (samples,), generator=gc).to(I32).cuda()
            q, k, v = rand(samples, N, Hq, D), rand(samples, N, Hkv, D), rand(samples, N, Hkv, D)
        o, lens = torch.empty_like(q), cache.lens.clone()
        if workspace is None:      # the same sizes at every step
            workspace = gdn.attn_workspace(q, cache.pool[0], cache.table, prefix)
        granted = cache.window(q, k, v, o, samples, parent, prefix, workspace, pass_in=into)
        if choice:
            more = choice.step(parent, granted)
            node = choice.node.clone()
        now, x = sets[i % 2], rand(samples, N, wl.C, t=io)
        og = torch.empty(samples, N, wl.Hv, wl.dv, dtype=io, device="cuda")
        gdn.verify_tree_step(x, w, parent, rand(samples, N, wl.Hv, t=io), rand(samples, N, wl.Hv, t=io), dt_bias, A_log,
                             now["H"], og, torch.empty_like(x), wl.Hk, S_prev, hist_prev, prev=prev, S_ckpt=now["S"],
                             hist_out=now["hist"])
        cache.accept(node, parent, granted, samples)
        S_prev, hist_prev, prev = now["S"], now["hist"], (node, parent, now["H"], x)
        windows.append(dict(q=q, k=k, v=v, o=o, og=og, parent=parent, node=node, lens=lens, granted=granted, **more))

    record = dict(prompt=kept, windows=windows, prefix=prefix, freed=list(range(1, samples, 2)), full_lens=cache.lens.clone())
    if choice:
        record.update(text=choice.history, text_lens=choice.lens, text_start=choice.start, params=choice.params)
    if record["freed"]:
        gdn.kv_free(torch.tensor(record["freed"], dtype=I32, device="cuda"), cache.lens, cache.table, cache.ref)
    cache.compact()
    return cache, record


def main():
    for vocab in (0, 32000):
        cache, record = run(vocab=vocab)
        torch.cuda.synchronize()
        took = [int(x) for x in record["full_lens"]]
        print("samples of %d tokens after %d tree steps behind a shared prefix of %d; after freeing %s: %d of %d pages in "
              "use, all below page %d" % (max(took), len(record["windows"]), record["prefix"], record["freed"],
                                          int((cache.ref > 0).sum()), cache.ref.numel(), int(cache.table.max()) + 1))
        if vocab:
            print("the nodes accepted by their logits: %s" % [w["node"].tolist() for w in record["windows"]])


if __name__ == "__main__":
    main()
