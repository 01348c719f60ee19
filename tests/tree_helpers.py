"""Plain models of drafted trees for their tests: sets and depths by walking up,
greedy acceptance one node after another, attention of a tree in 64 bits."""
import random

import numpy as np

from paged_helpers import rows_of


def random_tree(r, nodes, used, roots=1):
    """Parents of a tree of `used` of `nodes` nodes."""
    p = [-1 if m < roots else r.randrange(m) for m in range(used)]
    return p + [-2] * (nodes - used)


def trees(seed, batch, nodes):
    """A batch of them: ragged, with chains, fans and unused nodes."""
    r = random.Random(seed)
    got = []
    for b in range(batch):
        used = nodes if b == 0 else r.randint(0, nodes)
        kind = b % 4
        if kind == 1:
            got.append([m - 1 for m in range(used)] + [-2] * (nodes - used))            # a chain
        elif kind == 2:
            got.append([-1 if m == 0 else 0 for m in range(used)] + [-7] * (nodes - used))   # a fan
        else:
            got.append(random_tree(r, nodes, used, roots=1 + (kind == 3)))
    return got


def sets_of(parents):
    """Of each node: (depth, the nodes that it sees from the top down); (-1, []) for one that is not used."""
    up = []
    for m, p in enumerate(parents):
        if p < -1 or p >= m or (p >= 0 and up[p][0] < 0):
            up.append((-1, []))
        else:
            up.append((0, [m]) if p < 0 else (up[p][0] + 1, up[p][1] + [m]))
    return up


def bits_of(parents, window=0):
    """uint32 [nodes][words]."""
    n = len(parents)
    out = np.zeros((n, -(-n // 32)), np.uint32)
    for m, (_, s) in enumerate(sets_of(parents)):
        for j in s[-window:] if window else s:
            out[m, j // 32] |= np.uint32(1 << (j % 32))
    return out


def accept(parents, tokens, logits, width):
    """(emitted tokens, nodes)."""
    ups = sets_of(parents)
    cur, out, path = (0 if ups[0][0] >= 0 else None), [], []
    while cur is not None and len(out) < width:
        t = int(np.argmax(logits[cur]))           # the first of the largest
        out.append(t)
        path.append(cur)
        cur = next((c for c in range(cur + 1, len(parents)) if parents[c] == cur and ups[c][0] >= 0 and tokens[c] == t), None)
    return out, path


def tree_attention64(hp, layer, table, q, lens, planes, scale, parents, softcap=0.0, window=0, slopes=None, gone=None):
    """(out, tol) as paged_helpers.attention64 derives them, over the rows that each node sees
    (less those that are gone[b])."""
    B, M, Hq, D = q.shape
    g = Hq // hp.H
    out, tol = np.zeros((B, M, Hq, D)), np.zeros((B, M, Hq, D))
    c = 2.0 ** -8 if hp.bf else 2.0 ** -11
    for b in range(B):
        n = int(lens[b])
        base = n - M
        if n == 0:
            continue
        K, V = rows_of(hp, layer, table[b], n, planes)
        for m, (d, up) in enumerate(sets_of(parents[b])):
            if d < 0:
                continue
            at = base + d
            rows = np.array(list(range(max(base, 0))) + [base + j for j in up if base + j >= 0], np.int64)
            pos = np.array(list(range(max(base, 0))) + [base + k for k, j in enumerate(up) if base + j >= 0], np.int64)
            seen = pos > at - (window or 1 << 40)         # (positions below 0 where a sequence is shorter than its tree)
            if gone is not None:
                seen &= ~gone[b][rows]
            rows, pos = rows[seen], pos[seen]
            if len(rows) == 0:
                continue
            for h in range(Hq):
                k, v = K[h // g, rows], V[h // g, rows]
                x = q[b, m, h].astype(np.float64)
                s = scale * (k @ x)
                e = 2.0 ** -17 * scale * (np.abs(k) @ np.abs(x)).max()
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                    e += 2.0 ** -21 * softcap
                if slopes is not None:
                    bias = float(slopes[h]) * (at - pos)
                    s = s - bias
                    e += 2.0 ** -22 * np.abs(bias).max()
                p = np.exp(s - s.max())
                l = p.sum()
                out[b, m, h] = p @ v / l
                near = p @ np.abs(v) / l
                tol[b, m, h] = (2.0 ** -8 * np.abs(out[b, m, h]) + (2 * c + 2 * e) * near
                                + len(p) * 2.0 ** -24 * np.abs(v).max() / l)
    return out, tol
