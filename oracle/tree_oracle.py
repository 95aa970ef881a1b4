"""The float64 oracle of a step with a tree of drafted tokens: its attention, which drafts stay, and the rows that move.

Conventions (``include/fdecode.h``): the m tokens of a sequence are its last m places and the last m of its n rows;
``parents`` holds, row by row, the number of a token's parent (below its own) or -1.
"""

import numpy as np


def ancestors(parents):
    """Truth values [m, m] of one sequence's tokens: j is an ancestor of i, or i itself."""
    m = len(parents)
    sees = np.eye(m, dtype=bool)
    for i in range(m):
        up = int(parents[i])
        while up >= 0:
            assert up < i
            sees[i, up] = True
            up = int(parents[up])
    return sees


def attend(q, k, v, parents, lens, new_lens, scale):
    """q [B, Hq, n, D], k and v [B, Hkv, T, D] in any type; out [B, Hq, n, D] and lse [B, Hq, n] in 64 bits, NaN in the
    padding rows."""
    B, Hq, n, D = q.shape
    Hkv = k.shape[1]
    g = Hq // Hkv
    out, lse = np.full((B, Hq, n, D), np.nan), np.full((B, Hq, n), np.nan)
    for b in range(B):
        L = int(lens[b])
        m = n if new_lens is None else min(n, max(0, int(new_lens[b])))
        if m == 0:
            continue
        sees = ancestors(parents[b, n - m:])
        for i in range(m):
            at = [t for t in range(max(0, L - m))]
            at += [L - m + j for j in range(m) if sees[i, j] and L - m + j >= 0]
            for h in range(Hq):
                row = n - m + i
                if not at:
                    out[b, h, row], lse[b, h, row] = 0.0, -np.inf
                    continue
                x = k[b, h // g, at].astype(np.float64) @ q[b, h, row].astype(np.float64) * scale
                top = x.max()
                e = np.exp(x - top)
                out[b, h, row] = e @ v[b, h // g, at].astype(np.float64) / e.sum()
                lse[b, h, row] = top + np.log(e.sum())
    return out, lse


def verify(tokens, parents, target, uniforms, draft=None):
    """One sequence's walk.  tokens, parents, uniforms [m]; target [m, V]; draft [m, V] or None (the drafts are given, not
    drawn).  Returns (numbers of the tokens that stay, the next token or -1)."""
    m = len(tokens)
    if m == 0:
        return [], -1
    node, path = 0, [0]
    while True:
        p, q = (None if x is None else np.where(x[node] > 0, x[node], 0).astype(np.float64) for x in (target, draft))  # NaN too
        left, mass = p.copy(), 1.0
        for child in [i for i in range(m) if parents[i] == node and i > node]:
            x, u = int(tokens[child]), float(uniforms[child])
            share = float(q[x]) if draft is not None else 1.0
            if u * mass * share < left[x]:
                path.append(child)
                node = child
                break
            if draft is not None:
                left = np.maximum(left - mass * q, 0.0)
                mass = left.sum()
            else:
                mass -= left[x]
                left[x] = 0.0
        else:
            if not left.sum() > 0:
                left = p
            if not left.sum() > 0:
                return path, -1
            sums = np.cumsum(left)
            found = int(np.searchsorted(sums, float(uniforms[0]) * sums[-1], side="right"))
            return path, min(found, int(np.nonzero(left > 0)[0][-1]))


def keep(x, index, starts, counts):
    """x [B, Hkv, T, D] with row starts[b] + j replaced by row starts[b] + index[b, j], for j < counts[b]."""
    y = x.copy()
    for b in range(x.shape[0]):
        s = int(starts[b])
        for j in range(int(counts[b])):
            y[b, :, s + j] = x[b, :, s + int(index[b, j])]
    return y
