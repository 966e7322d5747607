"""fp64 oracle of the calls on drafted trees: what a row sees, attention by visibility
words over the 8-bit cache, the test of the drafts, the rows that a commit appends.

Plain numpy from the definitions; it shares no code with the CUDA path.  Verification
keeps the residual distribution itself, normalised after each rejection, where the
kernel keeps one number for it.
"""
from __future__ import annotations

import numpy as np

from oracle import cache_oracle as co


def ancestors(parents):
    """[rows, rows] bool: row i sees row j (itself and its ancestors)."""
    n = len(parents)
    sees = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while j >= 0:
            sees[i, j] = True
            j = int(parents[j])
    return sees


def words(sees, width):
    """The rows of a bool matrix as int32 words of 32 bits, `width` to a row."""
    out = np.zeros((len(sees), width), np.int64)
    for i, j in zip(*np.nonzero(sees)):
        out[i, j // 32] |= 1 << (j % 32)
    return out.astype(np.uint32).view(np.int32)


def attn(c, Q, K, V, sees, offsets, scale):
    """co.attn with `sees`, a bool matrix for each sequence; values at hidden keys do not enter."""
    T, Hq, d = Q.shape
    g = Hq // c["k8"].shape[1]
    O, A = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    LSE, E = np.full((Hq, T), -np.inf), np.zeros((Hq, T))
    for s in range(len(c["lens"])):
        a, b = int(offsets[s]), int(offsets[s + 1])
        for hq in range(Hq if b > a else 0):
            ck, cv = co.tokens(c, "k", s, hq // g), co.tokens(c, "v", s, hq // g)
            for i in range(a, b):
                own = a + np.flatnonzero(sees[s][i - a])
                k, v = np.concatenate([ck, K[own, hq // g]]), np.concatenate([cv, V[own, hq // g]])
                if len(k) == 0:
                    continue
                q = Q[i, hq].astype(np.float64)
                z = k @ q * scale
                p = np.exp(z - z.max())
                LSE[hq, i] = z.max() + np.log(p.sum())
                O[i, hq], A[i, hq] = p / p.sum() @ v, p / p.sum() @ np.abs(v)
                E[hq, i] = (np.abs(k) @ np.abs(q) * scale).max()
    return O, LSE, A, E


def verify(parents, tokens, target, draft, uniforms, sample, max_path):
    """(path, next token) of one sequence's tree; target, draft [rows, V]."""
    if len(parents) == 0:
        return [], -1
    V = target.shape[1]
    target = np.clip(np.nan_to_num(target.astype(np.float64), nan=0.0), 0, 1)
    draft = None if draft is None else np.clip(np.nan_to_num(draft.astype(np.float64), nan=0.0), 0, 1)
    path = [0]
    while True:
        cur = path[-1]
        p = target[cur]
        r, left, lost = p.copy(), 1.0, []  # what p has left, its total, the rejected tokens
        nxt = None
        kids = [j for j in range(1, len(parents)) if parents[j] == cur and 0 <= tokens[j] < V]
        for j in kids if len(path) < max_path else []:
            x, u = int(tokens[j]), float(uniforms[j])
            if draft is not None:
                if u * draft[cur, x] < r[x]:
                    nxt = j
                    break
                r = np.maximum(r - draft[cur], 0.0)
                if r.sum() > 0:
                    r = r / r.sum()
            else:
                if x not in lost and u * left < p[x]:
                    nxt = j
                    break
                if x not in lost:
                    lost.append(x)
                    left -= p[x]
                    r[x] = 0.0
        if nxt is None:
            break
        path.append(nxt)
    if r.sum() == 0:
        r = p
    if r.sum() == 0:
        return path, -1
    cdf = np.cumsum(r)
    return path, int(np.flatnonzero(cdf > float(sample) * cdf[-1])[0])


def commit(c, K, V, path, accepted, offsets):
    """Writes the accepted rows into c; returns the new lengths."""
    rows = [int(offsets[s]) + int(r) for s in range(len(accepted)) for r in path[s][: int(accepted[s])]]
    return co.append(c, K[rows], V[rows], np.concatenate([[0], np.cumsum(accepted)]))
