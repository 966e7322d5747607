"""The calls on drafted trees at the ends of their ranges: the largest trees, more own rows than a tree has, random
numbers outside [0, 1), two captured steps that share their workspaces.  Compared as in test_gpu_tree.py."""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle.tree_oracle as to
from tests.cache_util import device_cache, make_cache, make_rows, offsets_of
from tests.test_gpu_cache import check_attn, lib  # noqa: F401
from tests.test_gpu_tree import DEV, run_verify, step_inputs, verify_step
from tests.test_gpu_tree_tiles import attend, batch
from tests.tree_plain import plain_attn
from tests.tree_util import make_drafts, make_tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kids", [1, 4])
@pytest.mark.parametrize("drawn", [True, False])
def test_verify_the_largest_trees(lib, kids, drawn):
    """4096 rows; drawn drafts are near the target, so that paths are long.  (Chosen ones are accepted as often as the
    target draws them, a third of the time here, and in the second call, of steep distributions, nearly always.)"""
    ws, got = run_verify(lib, [4096, 10, 4095], kids, 40, drawn, seed=kids, near=0.02)
    lib.bdlm_sync_status(ws)
    if drawn:
        assert max(got[1]) > (10 if kids == 1 else 3)
    run_verify(lib, [4096, 10, 4095], kids, 40, drawn, seed=kids, near=0.02, spread=40.0)


def test_verify_random_numbers_out_of_range(lib):
    """NaN and numbers below 0 (-0 too) count as 0."""
    m = lib
    trees = [make_tree(12, 3, i) for i in range(8)]
    parents, tokens, target, draft, u, s = make_drafts(trees, 30, 3)
    target[:, ::4] = 0  # (0 is not below 0: such drafts are rejected whatever their number)
    bad = np.asarray([math.nan, -1.0, -0.0, -math.inf], np.float32)
    low, high = np.zeros_like(u), np.zeros_like(s)
    for q in (draft, None):
        d = None if q is None else DEV(q)
        call = lambda u, s: m.bdlm_tree_verify(DEV(parents), DEV(tokens), DEV(target), d, DEV(u), DEV(s))
        want = call(low, high)
        for shift in range(4):
            got = call(np.resize(np.roll(bad, shift), u.shape), np.resize(np.roll(bad, shift), s.shape))
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("d,o_dtype", [(64, torch.bfloat16), (128, torch.float32)])
@pytest.mark.parametrize("spoiled", [False, True])
def test_attn_more_rows_than_a_tree_has(lib, d, o_dtype, spoiled):
    """4500 own rows (36 tiles of keys), each seeing 40 of them; rows that none sees hold large values."""
    n = 4500
    x = batch([200], [n], 1, 1, d, 64, 7)
    i = np.arange(n)
    see = np.zeros((n, n), bool)
    for k in range(40):
        see[i, (i * 7 + k * 113) % n] = True
    see[:, 5::9] = False
    ref = plain_attn(torch, *(x[j] for j in (0, 2, 3, 4)), [see], x[1], 1 / math.sqrt(d))
    if spoiled:
        x[4][5::9] = np.resize(np.asarray([1e30, math.nan, -math.inf, 1e10], np.float32), len(x[4][5::9]))[:, None, None]
    O, LSE = attend(lib, *x, [see], o_dtype)
    check_attn(O, LSE, ref, d, o_dtype == torch.bfloat16)


def test_two_captured_steps_share_their_workspaces(lib):
    """Replayed in turn, each on its own cache and trees: as the calls made one by one.  (Positions stay below the 256
    that step_inputs has: after three steps lengths are at most 192 for 64 rows, 160 for the others.)"""
    m = lib
    rows = [[12, 7, 3, 20], [1, 64, 9, 5]]
    make = lambda: device_cache(m, torch, make_cache([40, 0, 100, 77], 256, 2, 64, 16, seed=1)[0])
    ws, vws = m.bdlm_cache_workspace(make(), 4, 64), m.bdlm_verify_workspace(4, 64, 211)
    xs = [step_inputs(3 + i, r)[0] for i, r in enumerate(rows)]
    side = torch.cuda.Stream()
    caches, graphs, outs = [make(), make()], [], []
    with torch.cuda.stream(side):
        for x in xs:
            verify_step(m, make(), x, ws, vws)
    torch.cuda.synchronize()
    for c, x in zip(caches, xs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = verify_step(m, c, x, ws, vws)
            c.lens.copy_(y["lens"])
        graphs.append(g)
        outs.append(y)
    plain = [make(), make()]
    for _ in range(3):
        for i in (0, 1):
            graphs[i].replay()
            z = verify_step(m, plain[i], xs[i], m.bdlm_cache_workspace(plain[i], 4, 64), m.bdlm_verify_workspace(4, 64, 211))
            plain[i].lens.copy_(z["lens"])
            for k in z:
                assert torch.equal(outs[i][k], z[k]), (i, k)
    for i in (0, 1):
        assert torch.equal(caches[i].k8.view(torch.uint8), plain[i].k8.view(torch.uint8))
        assert torch.equal(caches[i].lens, plain[i].lens)
    m.bdlm_sync_status(ws)
    m.bdlm_sync_status(vws)
