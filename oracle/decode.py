"""The decoding operators (masks of drafted trees, attention over a tree,
sampling, acceptance, the cache's move) from their definitions, in 64 bits or
more.

TEST INFRASTRUCTURE ONLY (same rules as the rest of this package): torch and
numpy on the CPU, straight from the formulas; shares no code with the HIP
library.
"""
from __future__ import annotations

import math

import numpy as np
import torch

F64 = torch.float64


def ancestors(parents):
    """[n] parents of one tree -> (bool [n, n]: row i sees i and its ancestors, depths)."""
    n = len(parents)
    see = np.zeros((n, n), dtype=bool)
    depth = [0] * n
    for i, p in enumerate(parents):
        if 0 <= p < i:
            see[i] = see[p]
            depth[i] = depth[p] + 1
        see[i, i] = True
    return see, depth


def words_of(see, words):
    """bool [rows, n] -> int32 words [rows, words], bit j % 32 of word j / 32."""
    rows, n = see.shape
    out = np.zeros((rows, words), dtype=np.uint32)
    for j in range(min(n, 32 * words)):
        out[:, j // 32] |= see[:, j].astype(np.uint32) << np.uint32(j % 32)
    return torch.from_numpy(out.view(np.int32))


def accept(tokens, parents, sampled, max_path):
    """(path, next token) of one tree."""
    if not len(tokens):
        return [], -1
    path = [0]
    while len(path) < max_path:
        at = path[-1]
        child = [i for i in range(at + 1, len(tokens)) if parents[i] == at and tokens[i] == sampled[at]]
        if not child:
            break
        path.append(child[0])
    return path, sampled[path[-1]]


def compact(cache, table, seq_len, nodes, path):
    """Moves one sequence's path in an oracle.layer.Cache (bytes), all reads first."""
    moves = []
    keys = len(table) * cache.size
    prefix = min(max(seq_len, 0), keys) - nodes
    for j, node in enumerate(path):
        if not j <= node < nodes or prefix + j < 0:
            continue
        ends = []
        for t in (prefix + node, prefix + j):
            page = int(table[t // cache.size])
            ends.append((page, t % cache.size) if 0 <= page < cache.pages else None)
        if None in ends:
            continue
        (fp, ft), to = ends
        moves.append((to, [cache.bytes[fp][:, at].clone() for at in cache._places(ft)]))
    for (page, t), parts in moves:
        for at, part in zip(cache._places(t), parts):
            cache.bytes[page][:, at] = part


def attention_tree(q, cache, table, seq_lens, starts, see, scale, window=0):
    """q [total, hq, D]; see: per sequence bool [its nodes, its nodes].
    -> out, lse, the sum of p times the magnitude of the uncentred value, the
    score error bound (as oracle.layer.attention)."""
    total, hq, d = q.shape
    hkv = cache.hkv
    group = hq // hkv
    out = torch.zeros(total, hq, d, dtype=F64)
    size = torch.zeros(total, hq, d, dtype=F64)
    lse = torch.full((total, hq), -math.inf, dtype=F64)
    delta = torch.zeros(total, hq, dtype=F64)
    for b, n in enumerate(seq_lens):
        q0, q1 = starts[b], starts[b + 1]
        nodes = q1 - q0
        n = min(max(n, 0), table.shape[1] * cache.size)
        if nodes <= 0 or n == 0:
            continue
        base = n - nodes
        on = torch.zeros(nodes, n, dtype=torch.bool)
        if base > 0:
            on[:, :base] = True
        for j in range(max(0, -base), nodes):
            on[:, base + j] = see[b][:, j]
        if window:
            for i in range(nodes):
                at = torch.nonzero(on[i]).view(-1)
                on[i, at[: max(0, len(at) - window)]] = False
        page = table[b, torch.arange(n) // cache.size].long()
        there = (page >= 0) & (page < cache.pages)
        on &= there
        at = torch.nonzero(there).view(-1)
        if not len(at):
            continue
        rows = [cache.read(int(page[t]) * cache.size + int(t) % cache.size) for t in at]
        uk, sk, mk = (torch.stack([r[0][i] for r in rows], 1) for i in range(3))  # [hkv, n, D or 1]
        uv, sv, mv = (torch.stack([r[1][i] for r in rows], 1) for i in range(3))
        on = on[:, at]
        some = on.any(1)
        for h in range(hq):
            k = h // group
            x = q[q0:q1, h].to(F64)
            z = (x @ (uk[k] * sk[k] + mk[k]).t()) * scale
            z = z.masked_fill(~on, -math.inf)
            lse[q0:q1, h] = torch.logsumexp(z, 1)
            p = torch.softmax(z, 1).masked_fill(~some[:, None], 0.0)
            out[q0:q1, h] = p @ (uv[k] * sv[k] + mv[k])
            size[q0:q1, h] = p @ (uv[k] * sv[k] + mv[k].abs())
            most = torch.where(on, (15 * sk[k] + mk[k].abs()).view(1, -1), torch.zeros(1, dtype=F64)).amax(1)
            top = torch.where(on, sk[k].view(1, -1), torch.zeros(1, dtype=F64)).amax(1)
            zmax = torch.where(on, z, torch.zeros(1, dtype=F64)).abs().amax(1)
            delta[q0:q1, h] = (d * 2.0 ** -14 * x.abs().amax(1) * top * abs(scale) + 2.0 ** -21 * x.abs().sum(1) * most * abs(scale)
                               + 2.0 ** -22 * zmax)
    return out, lse, size, delta


def sample(x, u, t=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row of logits (float32 values, as they are held) -> (token, log of
    the probability with which it is drawn, margin: how far, relative to the
    kept weights, the nearest border of a choice lies).  80-bit numbers."""
    x = np.asarray(x, dtype=np.float32).astype(np.longdouble)
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        x = np.where(np.isnan(x), -np.inf, x)
        top = x.max()
        if top == -np.inf:
            return -1, -math.inf, math.inf
        first = int(np.argmax(x))
        if not t > 0:
            return first, 0.0, math.inf
        t = min(float(t), float(np.finfo(np.float32).max))
        w = np.where(x == top, 1, np.exp((x - top) / np.longdouble(t)))
    w = np.where(x == -np.inf, 0, w)
    order = np.lexsort((np.arange(len(x)), -x))
    keep = order[: top_k] if top_k > 0 else order
    margin = math.inf
    if top_p < 1:
        v = w[keep]
        before = np.concatenate([[0], np.cumsum(v)[:-1]])
        stop = np.longdouble(max(top_p, 0.0)) * v.sum()
        on = before < stop
        on[0] = True
        margin = min(margin, float(np.abs(before[1:][v[1:] > 0] - stop).min() / v.sum()) if (v[1:] > 0).any() else math.inf)
        keep = keep[on]
    if min_p > 0:
        least = min(float(min_p), 1.0)
        off = np.abs(w[keep] - least)[w[keep] != 1]
        margin = min(margin, float(off.min()) if len(off) else math.inf)
        keep = keep[w[keep] >= least]
    keep = np.sort(keep)
    keep = keep[w[keep] > 0]
    sums = np.cumsum(w[keep])
    total = sums[-1]
    if not u < 1:
        at = len(keep) - 1
    else:
        goal = np.longdouble(max(u, 0.0)) * total
        at = min(int(np.searchsorted(sums, goal, side="right")), len(keep) - 1)
        if len(keep) > 1:
            margin = min(margin, float(np.abs(sums[:-1] - goal).min() / total))
    return int(keep[at]), float(np.log(w[keep[at]] / total)), margin
