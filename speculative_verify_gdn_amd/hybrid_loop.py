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
attention and the recurrence.  `python -m speculative_verify_gdn_amd.hybrid_loop`
runs it and prints what it did.
"""
from __future__ import annotations

import torch

from . import gdn, synth

I32 = torch.int32


class Cache:
    """The paged cache of one attention layer: pool [2][n_pages][Hkv][page][D], a table row and a length for each
    sequence, and the users of each page."""

    def __init__(self, rows, slots, n_pages, Hkv, page, D, dtype, device="cuda"):
        self.pool = torch.zeros(2, n_pages, Hkv, page, D, dtype=dtype, device=device)
        self.table = torch.full((rows, slots), -1, dtype=I32, device=device)
        self.lens = torch.zeros(rows, dtype=I32, device=device)
        self.ref = torch.zeros(n_pages, dtype=I32, device=device)
        self.page = page

    def window(self, q, k, v, o, rows, parent=None, prefix_len=0, workspace=None):
        """Room for a window of the first `rows` sequences, its keys and values in place, its attention in o."""
        K = q.shape[1]
        add = torch.full((rows,), K, dtype=I32, device=q.device)
        granted = torch.empty_like(add)
        lens, table = self.lens[:rows], self.table[:rows]
        gdn.kv_reserve(lens, add, table, self.ref, self.page, granted)
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


def run(samples=4, prompt=200, steps=5, N=8, Hq=8, Hkv=2, D=64, page=16, dtype=torch.bfloat16, seed=0):
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

    # the prompt, in row 0
    hist = torch.zeros(1, wl.W - 1, wl.C, dtype=io, device="cuda")
    S = torch.zeros(1, wl.Hv, wl.dv, wl.dk, device="cuda")
    kept = []                      # keys and values of the tokens that row 0 committed
    for at in range(0, prompt, 64):
        K = min(64, prompt - at)
        q, k, v = rand(1, K, Hq, D), rand(1, K, Hkv, D), rand(1, K, Hkv, D)
        granted = cache.window(q, k, v, torch.empty_like(q), rows=1)
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
        node = torch.randint(-1, N, (samples,), generator=gc).to(I32).cuda()
        q, k, v = rand(samples, N, Hq, D), rand(samples, N, Hkv, D), rand(samples, N, Hkv, D)
        o, lens = torch.empty_like(q), cache.lens.clone()
        if workspace is None:      # the same sizes at every step
            workspace = gdn.attn_workspace(q, cache.pool[0], cache.table, prefix)
        granted = cache.window(q, k, v, o, samples, parent, prefix, workspace)
        now, x = sets[i % 2], rand(samples, N, wl.C, t=io)
        og = torch.empty(samples, N, wl.Hv, wl.dv, dtype=io, device="cuda")
        gdn.verify_tree_step(x, w, parent, rand(samples, N, wl.Hv, t=io), rand(samples, N, wl.Hv, t=io), dt_bias, A_log,
                             now["H"], og, torch.empty_like(x), wl.Hk, S_prev, hist_prev, prev=prev, S_ckpt=now["S"],
                             hist_out=now["hist"])
        cache.accept(node, parent, granted, samples)
        S_prev, hist_prev, prev = now["S"], now["hist"], (node, parent, now["H"], x)
        windows.append(dict(q=q, k=k, v=v, o=o, og=og, parent=parent, node=node, lens=lens, granted=granted))

    record = dict(prompt=kept, windows=windows, prefix=prefix, freed=list(range(1, samples, 2)), full_lens=cache.lens.clone())
    if record["freed"]:
        gdn.kv_free(torch.tensor(record["freed"], dtype=I32, device="cuda"), cache.lens, cache.table, cache.ref)
    cache.compact()
    return cache, record


def main():
    cache, record = run()
    torch.cuda.synchronize()
    took = [int(x) for x in record["full_lens"]]
    print("samples of %d tokens after %d tree steps behind a shared prefix of %d; after freeing %s: %d of %d pages in use, "
          "all below page %d" % (max(took), len(record["windows"]), record["prefix"], record["freed"],
                                 int((cache.ref > 0).sum()), cache.ref.numel(), int(cache.table.max()) + 1))


if __name__ == "__main__":
    main()
