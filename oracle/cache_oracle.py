"""fp64 oracle of the 8-bit cache: the e4m3 block format, the write into the
pages, attention over them, the weight that cached tokens receive, eviction.

Plain numpy, one sequence and head at a time, from the definitions; it shares
no code with the CUDA path.  A cache is a dict of arrays: ``k8``, ``v8`` uint8
codes [n_pages, Hkv, page, d]; ``ks``, ``vs`` [n_pages, Hkv]; ``table``
[n_seqs, max_pages]; ``lens`` [n_seqs].
"""
from __future__ import annotations

import math

import numpy as np


def _codes():
    v = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        x = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v[b] = math.nan if (b & 127) == 127 else -x if b & 128 else x
    return v


E4M3 = _codes()                    # value of each code
_POS = E4M3[:127]                  # 0 .. 448, ascending


def encode(x):
    """Nearest code (ties to the even code; beyond 448: 448; NaN: 127)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(_POS, np.nan_to_num(a), side="left")
    lo = np.maximum(hi - 1, 0)
    dl, dh = np.nan_to_num(a) - _POS[lo], _POS[hi] - np.nan_to_num(a)
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.isnan(x), 127, c)
    return (c + 128 * np.signbit(x)).astype(np.uint8)


def block_scale(values):
    """Smallest power of two >= 2^-64 that holds the magnitudes within 448."""
    amax = np.abs(values).max() if np.size(values) else 0.0
    if not np.isfinite(amax):
        return math.nan
    k = -64
    while 448.0 * 2.0 ** k < amax:
        k += 1
    return 2.0 ** k


def tokens(c, which, s, h, n=None):
    """fp64 values of the first n (default: all cached) tokens of sequence s."""
    n = int(c["lens"][s]) if n is None else n
    page = c["k8"].shape[2]
    out = np.zeros((n, c["k8"].shape[3]))
    for i in range(n):
        p = c["table"][s, i // page]
        out[i] = E4M3[c[which + "8"][p, h, i % page]] * float(c[which + "s"][p, h])
    return out


def append(c, K, V, offsets):
    """Writes new tokens into c's codes and scales; returns the new lengths."""
    page, Hkv = c["k8"].shape[2], c["k8"].shape[1]
    lens = c["lens"].copy()
    for s in range(len(lens)):
        L, n = int(c["lens"][s]), int(offsets[s + 1] - offsets[s])
        for j in range(L // page, -(-(L + n) // page)):
            a, b = max(L, j * page), min(L + n, (j + 1) * page)
            if a >= b:
                continue
            p = c["table"][s, j]
            for X, w in ((K, "k"), (V, "v")):
                for h in range(Hkv):
                    new = X[offsets[s] + a - L: offsets[s] + b - L, h].astype(np.float64)
                    scale, old = block_scale(new), a - j * page
                    if old:
                        was = float(c[w + "s"][p, h])
                        scale = math.nan if math.isnan(was) or math.isnan(scale) else max(scale, was)
                        if scale != was:
                            c[w + "8"][p, h, :old] = encode(E4M3[c[w + "8"][p, h, :old]] * was / scale)
                    c[w + "8"][p, h, old: old + b - a] = encode(new / scale)
                    c[w + "s"][p, h] = scale
        lens[s] = L + n
    return lens


def attn(c, Q, K, V, offsets, scale):
    """(O, LSE, A, E): output, log-sum-exp, and for tolerances A = sum_j p_ij |v_j|
    per output and E = max_j scale * sum |q_i k_j| per row."""
    T, Hq, d = Q.shape
    g = Hq // c["k8"].shape[1]
    O, A = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    LSE, E = np.full((Hq, T), -np.inf), np.zeros((Hq, T))
    for s in range(len(c["lens"])):
        a, b = int(offsets[s]), int(offsets[s + 1])
        if a == b:
            continue
        for hq in range(Hq):
            k, v = tokens(c, "k", s, hq // g), tokens(c, "v", s, hq // g)
            if K is not None:
                k, v = np.concatenate([k, K[a:b, hq // g]]), np.concatenate([v, V[a:b, hq // g]])
            if len(k) == 0:
                continue
            q = Q[a:b, hq].astype(np.float64)
            z = q @ k.T * scale
            m = z.max(1, keepdims=True)
            p = np.exp(z - m)
            tot = p.sum(1, keepdims=True)
            LSE[hq, a:b] = (m + np.log(tot))[:, 0]
            O[a:b, hq], A[a:b, hq] = p / tot @ v, p / tot @ np.abs(v)
            E[hq, a:b] = (np.abs(q) @ np.abs(k).T * scale).max(1)
    return O, LSE, A, E


def weights(c, Q, LSE, offsets, scale, W):
    """W plus the attention weight of each cached token, and the row bound E of attn."""
    W = W.astype(np.float64).copy()
    g = Q.shape[1] // c["k8"].shape[1]
    worst = 0.0
    for s in range(len(c["lens"])):
        a, b, n = int(offsets[s]), int(offsets[s + 1]), int(c["lens"][s])
        for hq in range(Q.shape[1] if b > a and n else 0):
            q, k = Q[a:b, hq].astype(np.float64), tokens(c, "k", s, hq // g)
            live = np.isfinite(LSE[hq, a:b])
            z = q @ k.T * scale
            W[s, hq // g, :n] += np.exp(z - LSE[hq, a:b].astype(np.float64)[:, None])[live].sum(0)
            worst = max(worst, (np.abs(q) @ np.abs(k).T * scale).max())
    return W, worst


def evict(c, W, dst, keep, sinks, recent):
    """Moves the kept tokens into the pages of dst; returns (lens, weights, kept)."""
    n_seqs, Hkv, cap = W.shape
    page = c["k8"].shape[2]
    lens, Wout = c["lens"].copy(), np.zeros_like(W)
    kept = np.full((n_seqs, Hkv, keep), -1, np.int32)
    for s in range(n_seqs):
        n = int(c["lens"][s])
        lens[s] = min(n, keep)
        for h in range(Hkv):
            rank = [(math.inf if i < sinks or i >= n - recent or math.isnan(W[s, h, i]) else float(W[s, h, i]))
                    for i in range(n)]
            best = sorted(sorted(range(n), key=lambda i: (i >= sinks and i < n - recent, -rank[i], i))[:keep])
            kept[s, h, : len(best)] = best
            Wout[s, h, : len(best)] = W[s, h, best]
            for w in ("k", "v"):
                x = tokens(c, w, s, h)[best]
                for j in range(-(-len(best) // page)):
                    part, p = x[j * page: (j + 1) * page], dst[s, j]
                    scale = block_scale(part)
                    c[w + "8"][p, h, : len(part)] = encode(part / scale)
                    c[w + "s"][p, h] = scale
    return lens, Wout, kept
