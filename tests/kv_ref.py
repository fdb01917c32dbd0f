"""Plain 64-bit forms of the paged cache calls and the window attention: Python
loops over CPU tensors, written from the statements in include/gdn.h."""
import math

import torch


def path(parent, i):
    """Nodes from the root to i (parents first; parent None: a chain)."""
    up = [i]
    while True:
        p = up[-1] - 1 if parent is None else int(parent[up[-1]])
        if not 0 <= p < up[-1]:
            return up[::-1]
        up.append(p)


def attn(q, kp, vp, lens, table, count=None, parent=None, scale=None):
    """o, lse in float64 and the three magnitudes that bound a float evaluation of each row: the number of keys,
    the weighted mean of |v| and the largest scale * sum |q||k|.  Rows past count are NaN."""
    B, K, Hq, D = q.shape
    n_pages, Hkv, page, _ = kp.shape
    P = table.shape[1]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    o = torch.full((B, K, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((B, K, Hq), math.nan, dtype=torch.float64)
    mean = torch.zeros(B, K, Hq, D, dtype=torch.float64)
    keys = torch.zeros(B, K, Hq, dtype=torch.float64)
    size = torch.zeros(B, K, Hq, dtype=torch.float64)
    for b in range(B):
        n = min(max(int(lens[b]), 0), P * page)
        w = K if count is None else min(max(int(count[b]), 0), K)
        pos = torch.arange(n + w)
        slot = pos // page
        ids = table[b].long()[slot.clamp(max=P - 1)]
        there = (slot < P) & (ids >= 0) & (ids < n_pages)
        for t in range(w):
            seen = there.clone()
            seen[n:] = False
            for j in path(None if parent is None else parent[b], t):
                if n + j < seen.numel():
                    seen[n + j] = there[n + j]
            at = pos[seen]
            for h in range(Hkv):
                heads = slice(h * G, (h + 1) * G)
                k = kp[ids[at], h, at % page].double()
                v = vp[ids[at], h, at % page].double()
                if at.numel() == 0:
                    o[b, t, heads], lse[b, t, heads] = 0, -math.inf
                    continue
                qq = q[b, t, heads].double()
                x = qq @ k.T * scale
                p = torch.softmax(x, -1)
                o[b, t, heads] = p @ v
                lse[b, t, heads] = torch.logsumexp(x, -1)
                mean[b, t, heads] = p @ v.abs()
                keys[b, t, heads] = at.numel()
                size[b, t, heads] = (qq.abs() @ k.abs().T * abs(scale)).amax(-1)
    return o, lse, keys, mean, size


def attn_bounds(o, lse, keys, mean, size, D, bf16):
    """How far a float evaluation may be off, counted from its roundings:
      x        a D-term sum and the scaling:          dx = (D + 4) 2^-23 size
      e^{x-m}  its argument (|x - m| <= 2 size) and the exponential: 2^-22 size + 2^-21
      weights  rounded to bf16 before the product with v (bf16 only): 2^-8
      sums     keys + 64 terms (64: joins of the parts)  (keys + 64) 2^-23
      o        its own rounding, 2^-8 or 2^-24 of |o|
    Each relative error of the weights counts twice, in the numerator and in the sum."""
    dx = (D + 4) * 2.0 ** -23 * size + 2.0 ** -22 * size + 2.0 ** -21
    rel = 2 * dx + 2 * (keys + 64) * 2.0 ** -23 + (2.0 ** -8 if bf16 else 0.0)
    to = mean * rel[..., None] + o.abs() * (2.0 ** -8 if bf16 else 2.0 ** -24) + 1e-30
    tl = dx + (keys + 64) * 2.0 ** -23 + lse.abs() * 2.0 ** -22
    return to, tl


def reserve(lens, add, table, ref, page):
    """Updates table [B][P] and ref (lists) in place; returns granted."""
    n = len(ref)
    granted = []
    free = [p for p in range(n) if ref[p] == 0]
    asked = 0
    start = len(free)
    for b, row in enumerate(table):
        ln = max(lens[b], 0)
        if add[b] <= 0 or (ln + add[b] - 1) // page >= len(row):
            granted.append(0)
            continue
        want = [s for s in range(ln // page, (ln + add[b] - 1) // page + 1) if not 0 <= row[s] < n]
        asked += len(want)
        if want and asked > start:
            granted.append(0)
            continue
        granted.append(add[b])
        for s in want:
            row[s] = free.pop(0)
            ref[row[s]] = 1
    return granted


def append(k, v, kp, vp, lens, table, count=None):
    B, K = k.shape[:2]
    n_pages, _, page, _ = kp.shape
    for b in range(B):
        for t in range(K if count is None else min(max(count[b], 0), K)):
            at = max(lens[b], 0) + t
            if at // page < len(table[b]) and 0 <= table[b][at // page] < n_pages:
                kp[table[b][at // page], :, at % page] = k[b, t]
                vp[table[b][at // page], :, at % page] = v[b, t]


def rollback(node, parent, lens, table, ref, pool, N, count=None):
    """Updates table, ref, pool in place; returns the new lengths."""
    n_pages, page = pool.shape[1], pool.shape[3]
    out = []
    for b, row in enumerate(table):
        ln = max(lens[b], 0)
        w = N if count is None else min(max(count[b], 0), N)
        keep = path(None if parent is None else parent[b], node[b]) if 0 <= node[b] < w else []
        for i, j in enumerate(keep):
            f, t = (ln + j) // page, (ln + i) // page
            if max(f, t) < len(row) and 0 <= row[f] < n_pages and 0 <= row[t] < n_pages:
                pool[:, row[t], :, (ln + i) % page] = pool[:, row[f], :, (ln + j) % page].clone()
        out.append(ln + len(keep))
        for s in range((out[-1] + page - 1) // page, len(row)):
            if 0 <= row[s] < n_pages:
                ref[row[s]] -= 1
                row[s] = -1
    return out


def free(rows, lens, table, ref):
    for r in rows:
        if 0 <= r < len(table):
            for s, p in enumerate(table[r]):
                if 0 <= p < len(ref):
                    ref[p] -= 1
                table[r][s] = -1
            lens[r] = 0


def fork(src, dst, lens, table, ref, pool):
    n_pages, page = pool.shape[1], pool.shape[3]
    unused = [p for p in range(n_pages) if ref[p] == 0]
    asked, start, granted = 0, len(unused), []
    old = list(lens)
    for a, b in zip(src, dst):
        fine = 0 <= a < len(table) and 0 <= b < len(table) and a != b
        if fine:
            ln = max(old[a], 0)
            full, part = divmod(ln, page)
            slots = full + (part > 0)
            fine = slots <= len(table[a]) and all(0 <= p < n_pages for p in table[a][:slots])
            fine = fine and not any(0 <= p < n_pages for p in table[b])
        if not fine:
            granted.append(0)
            continue
        asked += part > 0
        if part and asked > start:
            granted.append(0)
            continue
        granted.append(1)
        table[b] = table[a][:full] + [-1] * (len(table[a]) - full)
        for p in table[a][:full]:
            ref[p] += 1
        if part:
            table[b][full] = unused.pop(0)
            ref[table[b][full]] = 1
            pool[:, table[b][full]] = pool[:, table[a][full]]
        lens[b] = ln
    return granted


def compact(table, ref, pool):
    used = sum(r > 0 for r in ref)
    holes = [p for p in range(used) if ref[p] <= 0]
    moved = [p for p in range(used, len(ref)) if ref[p] > 0]
    out = [r if p < used and r > 0 else 0 for p, r in enumerate(ref)]
    for to, at in zip(holes, moved):
        pool[:, to] = pool[:, at]
        out[to] = ref[at]
    now = dict(zip(moved, holes))
    return [[now.get(p, p) for p in row] for row in table], out
