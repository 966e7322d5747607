"""What pins the oracle of the calls on drafted trees (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

import oracle.cache_oracle as co
import oracle.tree_oracle as to
from tests.cache_util import make_cache, make_rows, offsets_of
from tests.tree_util import make_probs, make_tree


def test_ancestors_of_a_tree_written_by_hand():
    sees = to.ancestors([-1, 0, 0, 1, -1])
    assert sees.astype(int).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 1, 0, 1, 0], [0, 0, 0, 0, 1]]
    assert to.words(sees, 2)[:, 0].tolist() == [1, 3, 5, 11, 16] and (to.words(sees, 2)[:, 1] == 0).all()
    far = np.zeros((1, 40), bool)
    far[0, [31, 33]] = True
    assert to.words(far, 2).tolist() == [[-2 ** 31, 2]]


def test_a_chain_is_causal_and_all_bits_are_the_block():
    """All rows visible: the cached attention's own block.  A chain: each row alone on a longer cache."""
    c, _ = make_cache([9, 0], 16, 1, 64, 16, seed=3)
    off = offsets_of([4, 3])
    Q, K, V = make_rows(7, 2, 64, 1), make_rows(7, 1, 64, 2), make_rows(7, 1, 64, 3)
    full = to.attn(c, Q, K, V, [np.ones((4, 4), bool), np.ones((3, 3), bool)], off, 0.125)
    for a, b in zip(full, co.attn(c, Q, K, V, off, 0.125)):
        assert np.allclose(a, b, atol=1e-13)
    chain = to.attn(c, Q, K, V, [to.ancestors(make_tree(n, 1, 0)) for n in (4, 3)], off, 0.125)
    last = co.attn(c, Q, K, V, off, 0.125)
    assert np.allclose(chain[0][[3, 6]], last[0][[3, 6]], atol=1e-13)  # the last rows see all
    first = co.attn(c, Q[[0, 4]], K[[0, 4]], V[[0, 4]], offsets_of([1, 1]), 0.125)
    assert np.allclose(chain[0][[0, 4]], first[0], atol=1e-13)


@pytest.mark.parametrize("kids,drawn", [(1, True), (2, True), (3, True), (1, False), (3, False)])
def test_tokens_follow_the_target(kids, drawn):
    """The first token behind row 0, over drafts and random numbers, is distributed as the target says: each of
    5 tokens within 5 standard deviations of its count."""
    rng = np.random.default_rng(kids + 10 * drawn)
    p, q = make_probs(1, 5, 1)[0], make_probs(1, 5, 2)[0]
    parents = np.r_[-1, np.zeros(kids, int)]
    target = np.concatenate([p[None], make_probs(kids, 5, 3)])
    draft = np.concatenate([q[None], make_probs(kids, 5, 4)])
    n, count = 20000, np.zeros(5)
    for _ in range(n):
        kid = rng.choice(5, kids, p=q / q.sum(dtype=float)) if drawn else np.argsort(-q)[:kids]
        tokens = np.r_[0, kid]
        path, nxt = to.verify(parents, tokens, target, draft if drawn else None, rng.random(kids + 1), rng.random(), 9)
        count[tokens[path[1]] if len(path) > 1 else nxt] += 1
    want = n * p.astype(float)
    assert (np.abs(count - want) <= 5 * np.sqrt(want * (1 - p))).all(), (count, want)


def test_chosen_drafts_are_the_drawn_ones_of_a_drafter_that_is_certain():
    """A drafter whose distribution is one token: chosen and drawn agree on a single child."""
    target = make_probs(2, 7, 5)
    draft = np.zeros((2, 7), np.float32)
    draft[0, 4] = 1
    for u in (0.0, 0.1, 0.5, 0.99):
        for s in (0.0, 0.3, 0.999):
            a = to.verify([-1, 0], [0, 4], target, draft, [0, u], s, 5)
            assert a == to.verify([-1, 0], [0, 4], target, None, [0, u], s, 5)


def test_path_is_cut_and_empty_trees_end():
    target = np.full((4, 4), 0.25, np.float32)
    draft = target.copy()
    path, nxt = to.verify([-1, 0, 1, 2], [0, 1, 2, 3], target, draft, [0.5] * 4, 0.6, 3)
    assert path == [0, 1, 2] and nxt == 2
    assert to.verify([], [], target[:0], None, [], 0.5, 3) == ([], -1)


def test_commit_is_an_append_of_the_rows_in_order():
    K, V = make_rows(6, 1, 64, 1), make_rows(6, 1, 64, 2)
    a, _ = make_cache([5, 17], 32, 1, 64, 16, seed=1)
    b = {k: v.copy() for k, v in a.items()}
    lens = to.commit(a, K, V, [[0, 2], [1, -1]], [2, 1], offsets_of([4, 2]))
    rows = [0, 2, 5]
    assert (lens == co.append(b, K[rows], V[rows], offsets_of([2, 1]))).all() and lens.tolist() == [7, 18]
    assert all((a[k] == b[k]).all() or k in ("ks", "vs") for k in a)
