"""Small drafted trees for the tests."""
from __future__ import annotations

import numpy as np


def make_tree(rows, kids, seed):
    """Parents of a random tree (kids = 1: a chain); row 0 is its only root."""
    rng = np.random.default_rng(seed)
    par, room = [-1], [kids]
    for i in range(1, rows):
        free = [j for j in range(i) if room[j]]
        j = free[-1] if kids == 1 else int(rng.choice(free))
        par.append(j)
        room[j] -= 1
        room.append(kids)
    return np.asarray(par[:rows], np.int32)


def make_probs(rows, V, seed, spread=2.0):
    """[rows, V] fp32 probabilities."""
    z = np.random.default_rng(seed).standard_normal((rows, V)) * spread
    e = np.exp(z - z.max(1, keepdims=True))
    return (e / e.sum(1, keepdims=True)).astype(np.float32)


def make_drafts(trees, V, seed, drawn=True, near=0.5, spread=2.0):
    """(parents, tokens, target, draft or None, uniforms, sample) of packed trees: tokens drawn from the draft's
    rows, or its likeliest ones in order."""
    rng = np.random.default_rng(seed)
    T = sum(len(t) for t in trees)
    z = rng.standard_normal((T, V)) * spread
    soft = lambda x: (lambda e: (e / e.sum(1, keepdims=True)).astype(np.float32))(np.exp(x - x.max(1, keepdims=True)))
    target, draft = soft(z), soft(z + rng.standard_normal((T, V)) * near)
    tokens = np.zeros(T, np.int32)
    at = 0
    for t in trees:
        rank = {}
        for i, p in enumerate(t):
            k = rank.get(p, 0)
            rank[p] = k + 1
            if p >= 0:
                q = draft[at + p].astype(np.float64)
                tokens[at + i] = rng.choice(V, p=q / q.sum()) if drawn else np.argsort(-q, kind="stable")[k % V]
        at += len(t)
    parents = np.concatenate(trees).astype(np.int32) if T else np.zeros(0, np.int32)
    return (parents, tokens, target, draft if drawn else None, rng.random(T, dtype=np.float32),
            rng.random(len(trees), dtype=np.float32))
