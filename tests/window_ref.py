"""Plain 64-bit forms of the rotary, logits and acceptance calls: loops over CPU
tensors, written from the statements in include/gdn.h."""
import math

import torch

from tests.kv_ref import path

H24, H53 = 2.0 ** -24, 2.0 ** -53          # half a step of 1 in 32 and in 64 bits


def positions(B, K, pos=None, lens=None, parent=None):
    """[B][K] positions as Python integers."""
    if pos is not None:
        return [[int(pos[b][t]) for t in range(K)] for b in range(B)]
    start = [0] * B if lens is None else [max(int(n), 0) for n in lens]
    return [[start[b] + (t if parent is None else len(path(parent[b], t)) - 1) for t in range(K)] for b in range(B)]


def turned(x, where, freqs, interleaved=False, mscale=1.0, w=None, eps=1e-6):
    """x [B][K][H][D] normed (with w) and turned, in float64, and how far a float32 evaluation may be off (before
    the rounding of the output): with h = 2^-24,
      the norm     D squares summed by at most 22 roundings one after the other (16 a lane in a chain, 6 joins),
                   halved by the root; mean, eps, root, reciprocal and two products one each: 11 + 6 = 17 h
      the turn     the part of half a turn as a float: h / 2 * 2 pi; sine and cosine within 2 units: 4 h; by mscale,
                   product, sum one each: 3 h; together below 11 h of (|a| + |b|)
      theta        three roundings of 64 bits."""
    B, K, H, D = x.shape
    half = freqs.numel()
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    off = (17.0 if w is not None else 0.0) * H24 * y.abs()
    out = y.clone()
    a, b = (torch.arange(half), torch.arange(half) + half) if not interleaved else (2 * torch.arange(half), 2 * torch.arange(half) + 1)
    theta = torch.tensor(where, dtype=torch.float64)[..., None] * freqs.double()
    c, s = (f(theta)[:, :, None, :] * mscale for f in (torch.cos, torch.sin))
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    size = (y[..., a].abs() + y[..., b].abs()) * abs(mscale)
    more = size * ((11.0 + (17.0 if w is not None else 0.0)) * H24 + 3 * H53 * theta.abs()[:, :, None, :])
    off[..., a] = more
    off[..., b] = more
    return out, off


def rounded(off, out, dtype):
    """The bound with the output's own rounding: half a step of it."""
    return off + (out.abs() + off) * (torch.finfo(dtype).eps / 2) + 1e-40


def logits(x, history=None, lens=None, start=None, tokens=None, parent=None, params=None, ids=None, values=None, mask=None,
           count=None):
    """[B][K][V] adjusted logits in float64 (rows past count NaN), and the same in float32, each step rounded once."""
    B, K, V = x.shape
    both = []
    for dt in (torch.float64, torch.float32):
        out = torch.full((B, K, V), math.nan, dtype=dt)
        for b in range(B):
            rep, presence, frequency, temp = (torch.tensor(1.0), torch.tensor(0.0), torch.tensor(0.0), torch.tensor(1.0)) if params is None else params[b]
            for t in range(K if count is None else min(max(int(count[b]), 0), K)):
                s, n = torch.zeros(V, dtype=torch.int64), torch.zeros(V, dtype=torch.int64)
                if params is not None:
                    if history is not None:
                        first = 0 if start is None else int(start[b])
                        for i in range(min(max(int(lens[b]), 0), history.shape[1])):
                            v = int(history[b, i])
                            if 0 <= v < V:
                                s[v] += 1
                                n[v] += i >= first
                    if tokens is not None:
                        for j in path(None if parent is None else parent[b], t):
                            v = int(tokens[b, j])
                            if 0 <= v < V:
                                s[v] += 1
                                n[v] += 1
                y = x[b, t].to(dt)
                y = torch.where(s > 0, torch.where(y > 0, y * (1 / rep.to(dt)), y * rep.to(dt)), y)
                y = torch.where(n > 0, y - (frequency.to(dt) * n.to(dt) + presence.to(dt)), y)
                if ids is not None:
                    last = {int(v): i for i, v in enumerate(ids[b])}
                    for v, i in last.items():
                        if 0 <= v < V:
                            y[v] = y[v] + values[b, i].to(dt)
                if mask is not None:
                    v = torch.arange(V)
                    y = torch.where((mask[b, t][v // 32] >> (v % 32)) & 1 > 0, y, torch.tensor(-math.inf, dtype=dt))
                if float(temp) >= 2.0 ** -126:
                    y = y * (1 / temp.to(dt))
                out[b, t] = y
        both.append(out)
    return both


def best(score):
    """The lowest index of the largest entry, -1 where every one is -inf or NaN."""
    rows = score.reshape(-1, score.shape[-1])
    rows = torch.where(rows.isnan(), -math.inf, rows)
    top = rows.amax(-1, keepdim=True)
    got = [(r == m).nonzero()[0, 0].item() if m > -math.inf else -1 for r, m in zip(rows, top)]
    return torch.tensor(got, dtype=torch.int32).view(score.shape[:-1])


def accept(target, tokens, parent=None, count=None, root=None, history=None, lens=None):
    """node, next, the new history rows and lengths, as lists."""
    B, K = len(target), len(target[0])
    nodes, nexts, rows, after = [], [], [], []
    for b in range(B):
        want = -1 if root is None else root[b]
        kept = []
        for i in range(K if count is None else min(max(count[b], 0), K)):
            up = path(None if parent is None else parent[b], i)
            good = want < 0 or tokens[b][up[0]] == want
            good = good and all(tokens[b][j] == target[b][p] and tokens[b][j] >= 0 for p, j in zip(up, up[1:]))
            if good and len(up) > len(kept):
                kept = up
        nodes.append(kept[-1] if kept else -1)
        nexts.append(target[b][kept[-1]] if kept else want if root is not None else -1)
        if history is not None:
            row = list(history[b])
            n = min(max(lens[b], 0), len(row))
            for i, j in enumerate(kept):
                if n + i < len(row):
                    row[n + i] = tokens[b][j]
            rows.append(row)
            after.append(min(n + len(kept), len(row)))
    return nodes, nexts, rows, after
