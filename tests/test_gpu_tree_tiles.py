"""Attention of drafted trees where a sequence's own rows fill several tiles of 128 keys, on the GPU
against 64 bits.

257 to 384 rows times heads of a group go in tiles of 128 rows: with one head to a KV head a sequence
then has three tiles of own keys, with two heads two, which the kernel's two halves take in turn.  With few
heads a CTA has a single tile of keys, with many whole sequences: both are run.
Tolerances: check_attn of test_gpu_cache.py.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle.tree_oracle as to
from tests.cache_util import device_cache, make_cache, make_rows, offsets_of
from tests.parity_util import to_dev
from tests.test_gpu_cache import check_attn, lib  # noqa: F401
from tests.test_gpu_tree import DEV, trees_of
from tests.tree_plain import plain_attn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def batch(lens, rows, g, Hkv, d, page, seed):
    c, _ = make_cache(lens, max(max(lens), 1), Hkv, d, page, seed)
    Q, K, V = (make_rows(sum(rows), H, d, seed + i + 1) for i, H in enumerate((g * Hkv, Hkv, Hkv)))
    return c, offsets_of(rows), Q, K, V


def attend(m, c, off, Q, K, V, sees, o_dtype):
    R = max(len(x) for x in sees)
    cache = device_cache(m, torch, c)
    ws = m.bdlm_cache_workspace(cache, Q.shape[1], R)
    vis = np.concatenate([to.words(x, -(-R // 32)) for x in sees])
    O, LSE = m.bdlm_attn_tree(*(to_dev(t, torch) for t in (Q, K, V)), DEV(vis), cache, DEV(off), R, o_dtype=o_dtype,
                              workspace=ws)
    m.bdlm_sync_status(ws)
    return O, LSE


@pytest.mark.parametrize("g,rows", [(1, [257, 129, 300]), (1, [300, 384, 5]), (1, [384, 1, 256]), (2, [129, 40, 160]),
                                    (2, [192, 150, 128])])
@pytest.mark.parametrize("lens", [[0, 0, 0], [100, 300, 0], [400, 1700, 130]])
@pytest.mark.parametrize("Hkv", [1, 24])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
def test_two_and_three_own_tiles(lib, g, rows, lens, Hkv, d, o_dtype):
    c, off, Q, K, V = batch(lens, rows, g, Hkv, d, 32, g + rows[0])
    sees = trees_of(rows, 3, sum(rows))
    ref = plain_attn(torch, c, Q, K, V, sees, off, 1 / math.sqrt(d))
    check_attn(*attend(lib, c, off, Q, K, V, sees, o_dtype), ref, d, o_dtype == torch.bfloat16)


@pytest.mark.parametrize("g,rows,at", [(1, 100, 50), (2, 150, 10), (2, 150, 140), (2, 192, 127), (1, 300, 10), (1, 300, 130),
                                       (1, 300, 299), (1, 384, 255), (2, 300, 70)])
@pytest.mark.parametrize("value", [math.nan, -math.inf])
@pytest.mark.parametrize("lens", [[0, 0, 0, 0], [100, 200, 300, 600]])
@pytest.mark.parametrize("Hkv", [1, 24])
@pytest.mark.parametrize("d,o_dtype", [(64, torch.bfloat16), (128, torch.float32)])
def test_values_that_are_not_finite_in_any_own_tile(lib, g, rows, at, value, lens, Hkv, d, o_dtype):
    """One value of one own row: rows that see it have an output that is not finite in its column and finite ones
    beside it, the others are as without it."""
    n = len(lens)
    c, off, Q, K, V = batch(lens, [rows] * n, g, Hkv, d, 32, rows)
    rng = np.random.default_rng(rows + at)
    sees, hide = [], []
    for s in range(n):
        x = rng.random((rows, rows)) < 0.5
        x[:, 0] = True
        sees.append(x)
        hide.append(x.copy())
        hide[s][:, at] = False
    ref = plain_attn(torch, c, Q, K, V, hide, off, 1 / math.sqrt(d))
    V[off[:-1] + at, :, 3] = value
    O, LSE = attend(lib, c, off, Q, K, V, sees, o_dtype)
    mark = np.concatenate([x[:, at] for x in sees])
    see, mine = np.flatnonzero(mark), np.flatnonzero(~mark)
    check_attn(O[mine], LSE[:, mine], (ref[0][mine], ref[1][:, mine], ref[2][mine], ref[3][:, mine]), d,
               o_dtype == torch.bfloat16)
    got = O[DEV(see)]
    assert not torch.isfinite(got[:, :, 3]).any()
    assert torch.isfinite(torch.cat([got[:, :, :3], got[:, :, 4:]], 2)).all()
    if math.isinf(value):
        assert (got[:, :, 3] == value).all()
