"""The calls on drafted trees on the GPU against the fp64 oracle.

Masks, positions, paths, tokens, codes, scales and lengths are equal.  Attention
has the tolerances of test_gpu_cache.py (check_attn): the weights and scores are
rounded in the same places, hidden keys add nothing.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle.cache_oracle as co
import oracle.tree_oracle as to
from tests.cache_util import device_cache, host_codes, make_cache, make_rows, offsets_of
from tests.parity_util import to_dev
from tests.test_gpu_cache import check_attn, lib  # noqa: F401
from tests.tree_util import make_drafts, make_tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda().to(torch.bfloat16)
DEV = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()


def small_cache(m, lens, page=16, Hkv=1, d=64, capacity=None, seed=1):
    c, _ = make_cache(lens, capacity or max(max(lens), 1), Hkv, d, page, seed)
    return c, device_cache(m, torch, c)


# -------------------------------------------------------------------- mask
@pytest.mark.parametrize("kids", [1, 2, 5])
@pytest.mark.parametrize("rows", [[1], [31, 32, 33], [0, 64, 5, 0, 100], [300, 257], [4096]])
def test_mask(lib, rows, kids):
    m = lib
    lens = [7 * i for i in range(len(rows))]
    c, cache = small_cache(m, lens, capacity=64)
    trees = [make_tree(n, kids, 3 + i) for i, n in enumerate(rows)]
    off, T, R = offsets_of(rows), sum(rows), max(rows)
    parents = np.concatenate(trees + [np.full(5, 77, np.int32)]).astype(np.int32)  # (rows behind the last sequence)
    W = -(-R // 32) + (1 if R < 4096 else 0)
    out = (torch.full((T + 5, W), 7, dtype=torch.int32, device="cuda"),
           torch.full((T + 5,), 7, dtype=torch.int32, device="cuda"))
    ws = m.bdlm_cache_workspace(cache)
    m.bdlm_tree_mask(cache, DEV(parents), DEV(off), R, out=out, workspace=ws)
    m.bdlm_sync_status(ws)
    vis, pos = (x.cpu().numpy() for x in out)
    for s, t in enumerate(trees):
        sees = to.ancestors(t)
        assert (vis[off[s]:off[s + 1]] == to.words(sees, W)).all()
        assert (pos[off[s]:off[s + 1]] == lens[s] + sees.sum(1) - 1).all()
    assert (vis[T:] == 7).all() and (pos[T:] == 7).all()


def test_mask_of_equal_trees_without_offsets_and_made_outputs(lib):
    m = lib
    c, cache = small_cache(m, [3, 5])
    t = [make_tree(6, 2, 1), np.asarray([-1, -1, 0, 1, 3, -1], np.int32)]  # (a forest too)
    vis, pos = m.bdlm_tree_mask(cache, DEV(np.concatenate(t)))
    want = [to.ancestors(x) for x in t]
    assert vis.shape == (12, 1) and (vis.cpu().numpy() == np.concatenate([to.words(w, 1) for w in want])).all()
    assert pos.tolist() == [int(3 + x) for x in want[0].sum(1) - 1] + [int(5 + x) for x in want[1].sum(1) - 1]


def test_mask_reports_parents_out_of_range(lib):
    m = lib
    c, cache = small_cache(m, [3])
    ws = m.bdlm_cache_workspace(cache)
    vis, pos = m.bdlm_tree_mask(cache, DEV(np.asarray([-1, 1, -5, 0, 40], np.int32)), workspace=ws)
    assert vis[:, 0].tolist() == [1, 2, 4, 9, 16] and pos.tolist() == [3, 3, 3, 4, 3]
    with pytest.raises(m.BdlmError, match="tree"):
        m.bdlm_sync_status(ws)
    m.bdlm_sync_status(ws)


# --------------------------------------------------------------- attention
def run_tree(m, lens, sees, Hq, Hkv, d, page, o_dtype=None, seed=0, extra=0, words=None, spoil=None, uniform=False):
    """sees: a bool matrix for each sequence.  spoil(K, V) may change what no row sees."""
    rows = [len(x) for x in sees]
    c, _ = make_cache(lens, max(max(lens), 1), Hkv, d, page, seed)
    off, n = offsets_of(rows), int(sum(rows))
    T = n + extra
    Q, K, V = (make_rows(T, H, d, seed + i + 1) for i, H in enumerate((Hq, Hkv, Hkv)))
    W = words or max(1, -(-max(rows) // 32))
    vis = np.concatenate([to.words(x, W) for x in sees] + [np.full((extra, W), -1, np.int32)])
    for s, r in enumerate(rows):  # bits of rows that the sequence does not have count for nothing
        for j in range(r, 32 * W):
            vis[off[s]:off[s + 1], j // 32] |= np.array(1 << (j % 32), np.uint32).astype(np.int32)
    ref = to.attn(c, Q[:n], K[:n], V[:n], sees, off, 1 / math.sqrt(d))
    if spoil:
        spoil(K, V, off)
    cache = device_cache(m, torch, c)
    ws = m.bdlm_cache_workspace(cache, Hq, max(rows))
    out = (torch.full((T, Hq, d), 7.0, dtype=o_dtype or torch.bfloat16, device="cuda"),
           torch.full((Hq, T), 7.0, dtype=torch.float32, device="cuda"))
    m.bdlm_attn_tree(*(to_dev(x, torch) for x in (Q, K, V)), DEV(vis), cache, None if uniform else DEV(off), max(rows),
                     out=out, workspace=ws)
    m.bdlm_sync_status(ws)
    check_attn(out[0][:n], out[1][:, :n], ref, d, out[0].dtype == torch.bfloat16)
    assert (out[0][n:] == 7).all() and (out[1][:, n:] == 7).all(), "rows behind the last sequence were touched"
    return out


def trees_of(rows, kids, seed=0):
    return [to.ancestors(make_tree(n, kids, seed + i)) for i, n in enumerate(rows)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [[1, 2, 5, 16, 3], [32, 31, 17, 0, 4], [60, 64, 33, 1, 0], [128, 129, 7, 200, 1]])
def test_attn_trees(lib, page, d, rows):
    """Tiles of 16 and 32 rows on mma.sync, 128 and 256 on tcgen05; empty caches, ends inside pages and tiles."""
    run_tree(lib, [0, 129, 300, 16, 77], trees_of(rows, 3, 5), 2, 1, d, page, seed=page + d, extra=3)


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (16, 8), (10, 2), (17, 1), (40, 8)])
@pytest.mark.parametrize("kids", [1, 4])
def test_attn_trees_head_groups(lib, Hq, Hkv, kids):
    run_tree(lib, [200, 77, 5], trees_of([9, 4, 13], kids), Hq, Hkv, 64, 16, seed=Hq)


@pytest.mark.parametrize("rows", [[5, 3], [20, 32], [64, 40], [130, 150], [300, 280]])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_attn_any_pattern(lib, rows, o_dtype, d):
    """Random bits, rows that see nothing of the own ones (with an empty cache: no key at all)."""
    rng = np.random.default_rng(sum(rows) + d)
    sees = [rng.random((n, n)) < 0.4 for n in rows]
    for x in sees:
        x[1] = False
        x[len(x) // 2] = False
    run_tree(lib, [0, 150], sees, 2, 1, d, 32, o_dtype=o_dtype, seed=4, words=-(-max(rows) // 32) + 2)


@pytest.mark.parametrize("rows", [6, 40, 140])
def test_attn_nothing_to_see_at_all(lib, rows):
    O, LSE = run_tree(lib, [0], [np.zeros((rows, rows), bool)], 2, 1, 64, 16)
    assert (O == 0).all() and torch.isneginf(LSE).all()


@pytest.mark.parametrize("rows", [[5, 3], [32, 20], [64, 50], [128, 100], [150, 300]])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
def test_attn_hidden_rows_hold_anything(lib, rows, value, o_dtype):
    """A third of the own rows is seen by none: their keys and values are not finite."""
    rng = np.random.default_rng(sum(rows))
    sees, hidden = [], []
    for n in rows:
        x = rng.random((n, n)) < 0.5
        h = np.arange(n) % 3 == 1
        x[:, h] = False
        sees.append(x)
        hidden.append(h)

    def spoil(K, V, off):
        for s, h in enumerate(hidden):
            K[off[s]:off[s + 1]][h] = value
            V[off[s]:off[s + 1]][h] = value

    run_tree(lib, [0, 210], sees, 4, 2, 64, 16, o_dtype=o_dtype, seed=9, spoil=spoil)


@pytest.mark.parametrize("rows,at", [(5, 2), (32, 17), (64, 40), (128, 127), (300, 10), (300, 299)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("what", ["K", "V"])
@pytest.mark.parametrize("L", [0, 500])
def test_attn_values_that_are_not_finite_reach_those_that_see_them(lib, rows, at, value, what, L):
    """One own row holds them: rows that see it have outputs that are not finite, the others are as without it."""
    m = lib
    d, Hq = 64, 2
    rng = np.random.default_rng(rows)
    x = rng.random((rows, rows)) < 0.5
    x[:, 0] = True
    sees = x[:, at].copy()
    hide = x.copy()
    hide[:, at] = False
    c, cache = small_cache(m, [L], capacity=max(L, 16))
    Q, K, V = (make_rows(rows, H, d, i + 1) for i, H in enumerate((Hq, 1, 1)))
    ref = to.attn(c, Q, K, V, [hide], offsets_of([rows]), 0.125)
    (K if what == "K" else V)[at, 0, 3 if what == "V" else slice(None)] = value
    O, LSE = m.bdlm_attn_tree(*(to_dev(t, torch) for t in (Q, K, V)), DEV(to.words(x, -(-rows // 32))), cache)
    mine = np.flatnonzero(~sees)
    if len(mine):
        check_attn(O[mine], LSE[:, mine], (ref[0][mine], ref[1][:, mine], ref[2][mine], ref[3][:, mine]), d, True)
    see = torch.from_numpy(np.flatnonzero(sees)).cuda()
    if what == "V":
        assert not torch.isfinite(O[see][:, :, 3]).any()
        rest = torch.cat([O[see][:, :, :3], O[see][:, :, 4:]], 2)
        assert torch.isfinite(rest).all()
        if math.isinf(value):
            assert (O[see][:, :, 3] == value).all()
    elif math.isnan(value):
        assert torch.isnan(O[see]).all()


def test_attn_long_prefix_spans_many_parts(lib):
    for rows in (4, 40, 200):
        run_tree(lib, [5000, 1], trees_of([rows, 2], 3), 4, 1, 64, 128, seed=9)


@pytest.mark.parametrize("rows", [[12, 9, 16], [16, 0, 13]])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("spoiled", [False, True])
def test_attn_32_rows_over_long_caches(lib, rows, d, o_dtype, spoiled):
    """17 to 32 rows and room for 65536 tokens (lengths up to 1500): both row tiles in each warp."""
    m = lib
    c, _ = make_cache([1500, 70, 0], 1500, 16, d, 128, seed=d)
    cap = np.zeros((3, 512), np.int32)
    cap[:, : c["table"].shape[1]] = c["table"]
    c["table"] = cap
    off, T = offsets_of(rows), sum(rows)
    Q, K, V = (make_rows(T, H, d, 2 + i) for i, H in enumerate((32, 16, 16)))
    sees = trees_of(rows, 3)
    if spoiled:  # the last row is seen by none but itself: its neighbours' results do not know of it
        for x in sees:
            if len(x):
                x[:, -1] = False
    ref = to.attn(c, Q, K, V, sees, off, 1 / math.sqrt(d))
    if spoiled:
        last = [int(off[s + 1]) - 1 for s, r in enumerate(rows) if r]
        K[last], V[last] = math.nan, math.inf
    vis = np.concatenate([to.words(x, 1) for x in sees])
    cache = device_cache(m, torch, c)
    O, LSE = m.bdlm_attn_tree(*(to_dev(x, torch) for x in (Q, K, V)), DEV(vis), cache, DEV(off), max(rows), o_dtype=o_dtype)
    check_attn(O, LSE, ref, d, o_dtype == torch.bfloat16)


@pytest.mark.parametrize("rows", [[53, 20, 52, 0, 3], [64, 64, 64, 52, 7], [110, 60, 103, 52, 20]])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
def test_attn_several_row_tiles(lib, rows, d, o_dtype):
    """5 heads to a KV head: one to three tiles of 256 rows, the last ones part empty."""
    run_tree(lib, [4200, 0, 130, 77, 600], trees_of(rows, 3), 5, 1, d, 32, o_dtype=o_dtype, seed=rows[0])


@pytest.mark.parametrize("rows", [1, 12, 20, 70])
@pytest.mark.parametrize("size", [2.0 ** 16, 2.0 ** 22, 2.0 ** 26])
def test_attn_scores_beyond_fp32s_fractions(lib, rows, size):
    """Scores of 2^20 and more: a row's LSE is its largest score, its output inside its values' range."""
    m = lib
    c, cache = small_cache(m, [700], seed=23)
    Q, K, V = (make_rows(rows, H, 64, 1 + i) for i, H in enumerate((2, 1, 1)))
    Q = (Q * np.float32(size)).astype(np.float32)
    sees = to.ancestors(make_tree(rows, 2, 1))
    ref = to.attn(c, Q, K, V, [sees], offsets_of([rows]), 0.125)
    for o_dtype in (torch.bfloat16, torch.float32):
        O, LSE = m.bdlm_attn_tree(*(to_dev(x, torch) for x in (Q, K, V)), DEV(to.words(sees, -(-rows // 32))), cache,
                                  o_dtype=o_dtype)
        assert torch.isfinite(O).all() and torch.isfinite(LSE).all()
        assert (np.abs(LSE.double().cpu().numpy() - ref[1])
                <= (64 + 8) * 2.0 ** -24 * ref[3] + 2.0 ** -21 + 2.0 ** -22 * np.abs(ref[1])).all()
        v = np.concatenate([co.tokens(c, "v", 0, 0), V[:, 0]])
        assert (O.double().cpu().numpy() <= v.max(0) * (1 + 2.0 ** -8) + 1e-3).all()
        assert (O.double().cpu().numpy() >= v.min(0) * (1 + 2.0 ** -8) - 1e-3).all()


@pytest.mark.parametrize("rows", [1, 12, 40, 200])
def test_attn_of_a_pool_past_32_bit_offsets(lib, rows):
    """Pages whose codes lie past 2^31 bytes (a pool of 2.4 GB for each of K and V, as good as empty)."""
    m = lib
    d, Hkv, page, n_pages = 128, 2, 128, 74000
    cc, _ = make_cache([300, 140], 384, Hkv, d, page, seed=4)
    far = np.asarray([[73999, 70001, 0], [65600, 1, 73111]], np.int32)  # the same pages, elsewhere
    c8 = {w: torch.zeros((n_pages, Hkv, page, d), dtype=torch.uint8, device="cuda") for w in "kv"}
    sc = {w: torch.ones((n_pages, Hkv), device="cuda") for w in "kv"}
    for s in range(2):
        for j in range(3):
            for w in "kv":
                c8[w][int(far[s, j])] = DEV(cc[w + "8"][cc["table"][s, j]])
                sc[w][int(far[s, j])] = DEV(cc[w + "s"][cc["table"][s, j]])
    cache = m.BdlmCache(c8["k"].view(torch.float8_e4m3fn), c8["v"].view(torch.float8_e4m3fn), sc["k"], sc["v"], DEV(far),
                        DEV(cc["lens"]))
    sees = trees_of([rows, rows], 2)
    Q, K, V = (make_rows(2 * rows, H, d, 1 + i) for i, H in enumerate((4, Hkv, Hkv)))
    vis = DEV(np.concatenate([to.words(x, -(-rows // 32)) for x in sees]))
    O, LSE = m.bdlm_attn_tree(*(to_dev(x, torch) for x in (Q, K, V)), vis, cache)
    off = offsets_of([rows, rows])
    check_attn(O, LSE, to.attn(cc, Q, K, V, sees, off, 1 / math.sqrt(d)), d, True)
    path = np.tile(np.arange(rows, dtype=np.int32), (2, 1))
    acc = np.asarray([rows, 1], np.int32)
    want = to.commit(cc, K, V, path, np.minimum(acc, [84, 84]) if rows > 84 else acc, off)
    ws = m.bdlm_cache_workspace(cache)
    got = m.bdlm_cache_commit(cache, to_dev(K, torch), to_dev(V, torch), DEV(path), DEV(acc), workspace=ws)
    if rows <= 84:  # (room for 84 more tokens)
        m.bdlm_sync_status(ws)
        assert got.tolist() == want.tolist()
        for s in range(2):
            for j in range(3):
                for w in "kv":
                    assert (c8[w][int(far[s, j])].cpu().numpy() == cc[w + "8"][cc["table"][s, j]]).all()


def test_attn_many_sequences(lib):
    run_tree(lib, [(37 * i) % 200 for i in range(70)], trees_of([1 + i % 4 for i in range(70)], 2), 4, 2, 64, 16, seed=11)


def test_attn_equal_trees_without_offsets(lib):
    run_tree(lib, [50, 90, 0], trees_of([8, 8, 8], 2), 4, 2, 64, 16, uniform=True, seed=5)


def test_attn_of_all_bits_is_cached_attention(lib):
    """Above 32 rows times heads of a group bit for bit: the same kernels, nothing hidden.  Up to 32 (4 rows here) the
    kernels are two, each off from the formula by check_attn's bound at most."""
    m = lib
    for rows in (4, 30, 64, 200):
        c, cache = small_cache(m, [700, 60], page=32, Hkv=2, d=128)
        Q, K, V = (to_dev(make_rows(2 * rows, H, 128, i + 1), torch) for i, H in enumerate((4, 2, 2)))
        vis = torch.full((2 * rows, -(-rows // 32)), -1, dtype=torch.int32, device="cuda")
        a, b = m.bdlm_attn_tree(Q, K, V, vis, cache), m.bdlm_attn_cached(Q, K, V, cache)
        if 2 * rows > 32:
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            continue
        ref = to.attn(c, *(make_rows(2 * rows, H, 128, i + 1) for i, H in enumerate((4, 2, 2))),
                      [np.ones((rows, rows), bool)] * 2, offsets_of([rows] * 2), 1 / math.sqrt(128))
        for x in (a, b):
            check_attn(x[0], x[1], ref, 128, True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [1, 8, 9, 16, 17, 24, 25, 32])
def test_attn_every_count_of_row_tiles(lib, rows, o_dtype, d):
    """Of 8 rows each, full and one over; caches split between CTAs and whole ones."""
    for lens in ([1500, 130], [900, 33]):
        run_tree(lib, lens, trees_of([rows, max(rows - 3, 1)], 3), 1, 1, d, 32, o_dtype=o_dtype, seed=rows)


@pytest.mark.parametrize("rows", [3, 13, 23, 31])
@pytest.mark.parametrize("d", [64, 128])
def test_attn_scores_that_climb(lib, rows, d):
    """Keys whose scores rise from tile to tile by less, about and more than a reference's step, and one row's by
    hundreds: references move often, and for one row of a warp's alone."""
    m = lib
    lens = [1400]
    c, _ = make_cache(lens, 1400, 1, d, 16, 7)
    Q, K, V = (make_rows(rows, 1, d, i + 1) for i in range(3))
    Q = Q / 8 + 1.0
    Q[rows // 2] *= 16
    Q = torch.from_numpy(Q.astype(np.float32)).to(torch.bfloat16).float().numpy()
    for b in range(-(-1400 // 16)):
        c["ks"][c["table"][0, b]] = 2.0 ** -12 * (1 + b / 4)
    sees = trees_of([rows], 2)
    off = offsets_of([rows])
    ref = to.attn(c, Q, K, V, sees, off, 1 / math.sqrt(d))
    cache = device_cache(m, torch, c)
    out = m.bdlm_attn_tree(*(to_dev(x, torch) for x in (Q, K, V)), DEV(np.concatenate([to.words(x, 1) for x in sees])),
                           cache, max_rows=rows)
    check_attn(out[0], out[1], ref, d, True)


@pytest.mark.parametrize("rows", [1, 40, 150])
def test_attn_reports_pages_and_lengths_out_of_range(lib, rows):
    m = lib
    c, _ = make_cache([100], 112, 1, 64, 16, seed=3)
    c["table"][0, 2] = 10 ** 6
    cache = device_cache(m, torch, c)
    Q, K, V = (to_dev(make_rows(rows, H, 64, i + 1), torch) for i, H in enumerate((2, 1, 1)))
    ws = m.bdlm_cache_workspace(cache, 2, rows)
    vis = DEV(to.words(to.ancestors(make_tree(rows, 2, 1)), -(-rows // 32)))
    O, LSE = m.bdlm_attn_tree(Q, K, V, vis, cache, workspace=ws)
    assert torch.isfinite(O).all()
    with pytest.raises(m.BdlmError, match="page id"):
        m.bdlm_sync_status(ws)


# ------------------------------------------------------------ verification
def run_verify(m, rows, kids, V, drawn=True, dtype=torch.float32, seed=0, max_path=None, pad=0, spoil=None, offsets=True,
               spread=2.0, near=0.5):
    trees = [make_tree(n, kids, seed + i) for i, n in enumerate(rows)]
    parents, tokens, target, draft, u, s = make_drafts(trees, V, seed, drawn, near, spread)
    if dtype == torch.bfloat16:
        target, draft = (None if x is None else torch.from_numpy(x).to(dtype).float().numpy() for x in (target, draft))
    if spoil:
        spoil(parents, tokens, target, draft, u, s)
    off, R = offsets_of(rows), max(max(rows), 1)
    wide = lambda x: None if x is None else torch.cat(
        [DEV(x).to(dtype), torch.full((len(x), pad), math.nan, dtype=dtype, device="cuda")], 1)[:, :V]
    ws = m.bdlm_verify_workspace(len(rows), R, V)
    path, acc, tok = m.bdlm_tree_verify(DEV(parents), DEV(tokens), wide(target), wide(draft), DEV(u), DEV(s),
                                        DEV(off) if offsets else None, R, max_path=max_path, workspace=ws)
    got = path.cpu().numpy(), acc.tolist(), tok.tolist()
    for i in range(len(rows)):
        a, b = off[i], off[i + 1]
        want, nxt = to.verify(parents[a:b], tokens[a:b], target[a:b], None if draft is None else draft[a:b], u[a:b], s[i],
                              max_path or R)
        assert got[1][i] == len(want) and got[2][i] == nxt, (i, got[1][i], want, got[2][i], nxt)
        assert got[0][i].tolist() == want + [-1] * (got[0].shape[1] - len(want))
    return ws, got


@pytest.mark.parametrize("V", [1, 2, 37, 1000, 4096, 20011])
@pytest.mark.parametrize("kids", [1, 3])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify(lib, V, kids, drawn, dtype):
    ws, got = run_verify(lib, [1, 8, 0, 30, 5, 64], kids, V, drawn, dtype, seed=V + kids)
    lib.bdlm_sync_status(ws)


@pytest.mark.parametrize("pad", [0, 1, 3, 5, 8])
@pytest.mark.parametrize("V", [129, 1003])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_rows_a_stride_apart(lib, pad, V, dtype):
    """Rows start anywhere in 16 bytes; what lies between them is NaN."""
    run_verify(lib, [9, 12, 7], 2, V, True, dtype, seed=pad + V, pad=pad)


def test_verify_rows_of_unlike_strides(lib):
    m = lib
    trees = [make_tree(12, 2, 1)]
    parents, tokens, target, draft, u, s = make_drafts(trees, 333, 8)
    a = torch.full((12, 340), math.nan, device="cuda")
    a[:, :333] = DEV(target)
    path, acc, tok = m.bdlm_tree_verify(DEV(parents), DEV(tokens), a[:, :333], DEV(draft), DEV(u), DEV(s))
    want, nxt = to.verify(parents, tokens, target, draft, u, s[0], 12)
    assert path[0, : len(want)].tolist() == want and acc.tolist() == [len(want)] and tok.tolist() == [nxt]


@pytest.mark.parametrize("n", [1, 3, 40, 100, 700])
def test_verify_clusters_of_any_size(lib, n):
    run_verify(lib, [1 + (5 * i) % 9 for i in range(n)], 2, 501, True, seed=n)


@pytest.mark.parametrize("kids,near", [(8, 0.5), (8, 3.0), (30, 3.0), (60, 4.0)])
@pytest.mark.parametrize("drawn", [True, False])
def test_verify_many_children(lib, kids, near, drawn):
    """Many children are rejected: c grows past whole numbers, totals shrink."""
    ws, got = run_verify(lib, [61] * 12, kids, 97, drawn, seed=kids, near=near)


@pytest.mark.parametrize("max_path", [1, 2, 3, 50])
def test_verify_path_is_cut(lib, max_path):
    run_verify(lib, [20, 9], 1, 300, True, seed=3, max_path=max_path, near=0.05)


def test_verify_equal_trees_without_offsets(lib):
    run_verify(lib, [7, 7, 7], 2, 100, True, seed=4, offsets=False)


@pytest.mark.parametrize("u", [0.0, 0.99999994])
@pytest.mark.parametrize("drawn", [True, False])
def test_verify_random_numbers_at_their_ends(lib, u, drawn):
    def spoil(parents, tokens, target, draft, us, s):
        us[:] = u
        s[:] = u
    run_verify(lib, [9, 12, 30], 3, 211, drawn, seed=5, spoil=spoil)


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_one_hot_rows(lib, drawn):
    """Greedy decoding: p is 1 at one token.  Where the draft's row is the same, all that it draws is accepted."""
    def spoil(parents, tokens, target, draft, us, s):
        best = target.argmax(1)
        target[:] = 0
        target[np.arange(len(target)), best] = 1
        if draft is not None:
            draft[:] = 0
            draft[np.arange(len(draft)), best] = 1
        at = 0
        for i in range(len(parents)):
            at = i if parents[i] < 0 else at
            if parents[i] >= 0 and i % 3:
                tokens[i] = best[at + parents[i]]
    run_verify(lib, [9, 16, 30], 3, 64, drawn, seed=6, spoil=spoil)


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_masked_vocabulary(lib, drawn):
    """Nine tokens in ten have probability 0 (the most likely ones were kept); drafts outside are rejected."""
    def spoil(parents, tokens, target, draft, us, s):
        for x in (target, draft):
            if x is not None:
                x[x < np.quantile(x, 0.9, axis=1, keepdims=True)] = 0
                x /= x.sum(1, keepdims=True)
        tokens[1::4] = 0
    run_verify(lib, [20, 33], 2, 500, drawn, seed=7, spoil=spoil)


def test_verify_the_same_token_twice(lib):
    """Children of one row with the same token: chosen, the second one is not accepted after the first; drawn,
    it is tested against what is left."""
    def spoil(parents, tokens, target, draft, us, s):
        tokens[:] = 3
    for drawn in (True, False):
        for seed in range(4):
            run_verify(lib, [9] * 20, 8, 6, drawn, seed=seed, spoil=spoil)


@pytest.mark.parametrize("total", [0.9, 1.1, 1.6])
@pytest.mark.parametrize("drawn", [True, False])
def test_verify_rows_that_do_not_sum_to_one(lib, total, drawn):
    """Chosen drafts may then use up more than 1: what is left falls below 0, and the next one is accepted."""
    def spoil(parents, tokens, target, draft, us, s):
        target *= np.float32(total)
        us[:] = 0.5 + us / 2
        tokens[:] = np.arange(len(tokens)) % 4
    for seed in range(5):
        run_verify(lib, [14] * 16, 6, 4, drawn, seed=seed, spoil=spoil, spread=0.3)


def test_verify_values_outside_their_range(lib):
    """NaN and below 0: 0; above 1: 1."""
    def spoil(parents, tokens, target, draft, us, s):
        target[:, 5] = math.nan
        target[:, 6] = -0.5
        draft[:, 7] = math.nan
        draft[:, 8] = 1.5
        tokens[2::3] = 5
        tokens[4::5] = 8
    run_verify(lib, [12, 9], 2, 40, True, seed=8, spoil=spoil)


def test_verify_leaves_bad_rows_out_and_says_so(lib):
    m = lib
    def spoil(parents, tokens, target, draft, us, s):
        tokens[3], tokens[5] = -1, 1000
    ws, got = run_verify(m, [12], 3, 50, True, seed=9, spoil=spoil)
    with pytest.raises(m.BdlmError, match="tree"):
        m.bdlm_sync_status(ws)
    m.bdlm_sync_status(ws)

    def spoil(parents, tokens, target, draft, us, s):
        target[:] = 0
    ws, got = run_verify(m, [12, 4], 3, 50, True, seed=9, spoil=spoil)
    assert got[2] == [-1, -1]
    with pytest.raises(m.BdlmError, match="tree"):
        m.bdlm_sync_status(ws)


def test_verify_reports_bad_offsets(lib):
    m = lib
    parents, tokens, target, draft, u, s = make_drafts([make_tree(4, 1, 0), make_tree(4, 1, 0)], 30, 1)
    ws = m.bdlm_verify_workspace(2, 4, 30)
    path, acc, tok = m.bdlm_tree_verify(DEV(parents), DEV(tokens), DEV(target), DEV(draft), DEV(u), DEV(s),
                                        DEV(np.asarray([0, 4, 9], np.int32)), 4, workspace=ws)
    assert acc[1] == 0 and tok[1] == -1 and (path[1] == -1).all() and acc[0] >= 1
    with pytest.raises(m.BdlmError, match="row offsets"):
        m.bdlm_sync_status(ws)


def test_verify_large_vocabulary_past_32_bit_offsets(lib):
    """Rows whose elements lie past 2^31 (bf16: 9 GB of rows that are mostly never looked at)."""
    m = lib
    V, T = 160000, 14000
    target = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    parents = np.full(T, -1, np.int32)
    parents[T - 4:] = [-1, 0, 1, 2]
    tokens = np.zeros(T, np.int32)
    target[T - 4, 7], target[T - 3, V - 1], target[T - 2, 5], target[T - 1, V - 2] = 1, 1, 1, 1
    tokens[T - 3:] = [7, V - 1, 4]
    off = np.asarray([T - 4, T, T, T], np.int32)
    z = torch.full((T,), 0.5, device="cuda")
    path, acc, tok = m.bdlm_tree_verify(DEV(parents), DEV(tokens), target, None, z, z[:3].clone(), DEV(off), 4)
    assert path[0].tolist() == [0, 1, 2, -1] and acc.tolist() == [3, 0, 0] and tok.tolist() == [5, -1, -1]


# ------------------------------------------------------------------ commit
def same(cache, c):
    for w in ("k", "v"):
        assert (host_codes(getattr(cache, w + "8")) == c[w + "8"]).all()
        np.testing.assert_array_equal(getattr(cache, w + "_scale").cpu().numpy(), c[w + "s"])


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_commit(lib, page, d):
    m = lib
    lens, rows = [0, 3, page - 1, page, 2 * page + 5, 40], [9, 4, 70, 0, 30, 5]
    acc = [4, 0, 33, 0, 30, 1]
    c, _ = make_cache(lens, max(lens) + 80, 3, d, page, seed=page)
    off, T = offsets_of(rows), sum(rows)
    rng = np.random.default_rng(d)
    K, V = (make_rows(T, 3, d, s) for s in (1, 2))
    path = np.full((6, 40), -1, np.int32)
    for s, a in enumerate(acc):
        path[s, :a] = np.sort(rng.permutation(rows[s])[:a]) if a else []
        path[s, a:] = 10 ** 6  # (not read)
    cache = device_cache(m, torch, c)
    ws = m.bdlm_cache_workspace(cache)
    want = to.commit(c, K, V, path, np.asarray(acc, np.int32), off)
    got = m.bdlm_cache_commit(cache, to_dev(K, torch), to_dev(V, torch), DEV(path), DEV(np.asarray(acc, np.int32)), DEV(off),
                              max(rows), workspace=ws)
    m.bdlm_sync_status(ws)
    assert got.tolist() == want.tolist()
    same(cache, c)


def test_commit_of_a_row_twice_and_out_of_order(lib):
    m = lib
    c, _ = make_cache([5], 48, 2, 64, 16, seed=2)
    K, V = (make_rows(6, 2, 64, s) for s in (1, 2))
    path = np.asarray([[4, 4, 0, 2, 4]], np.int32)
    cache = device_cache(m, torch, c)
    got = m.bdlm_cache_commit(cache, to_dev(K, torch), to_dev(V, torch), DEV(path), DEV(np.asarray([5], np.int32)))
    assert got.tolist() == to.commit(c, K, V, path, np.asarray([5]), offsets_of([6])).tolist()
    same(cache, c)


def test_commit_leaves_out_what_is_out_of_range(lib):
    m = lib
    c, _ = make_cache([5, 5, 5], 32, 1, 64, 16, seed=3)
    K, V = (make_rows(9, 1, 64, s) for s in (1, 2))
    path = np.asarray([[0, 7, -3], [0, 1, 2], [1, 0, 2]], np.int32)
    acc = np.asarray([3, 4, -1], np.int32)
    cache = device_cache(m, torch, c)
    ws = m.bdlm_cache_workspace(cache)
    got = m.bdlm_cache_commit(cache, to_dev(K, torch), to_dev(V, torch), DEV(path), DEV(acc), workspace=ws)
    assert got.tolist() == [8, 5, 5]
    with pytest.raises(m.BdlmError, match="tree"):
        m.bdlm_sync_status(ws)
    K2, V2 = (np.concatenate([x[:1], np.zeros((2, 1, 64), np.float32)]) for x in (K, V))
    co.append(c, K2, V2, offsets_of([3, 0, 0]))
    same(cache, c)


def test_commit_stops_at_the_end_of_the_table(lib):
    m = lib
    c, _ = make_cache([30], 32, 1, 64, 16, seed=4)
    K, V = (make_rows(6, 1, 64, s) for s in (1, 2))
    cache = device_cache(m, torch, c)
    ws = m.bdlm_cache_workspace(cache)
    got = m.bdlm_cache_commit(cache, to_dev(K, torch), to_dev(V, torch), DEV(np.asarray([[3, 1, 0, 5]], np.int32)),
                              DEV(np.asarray([4], np.int32)), workspace=ws)
    assert got.tolist() == [32]
    with pytest.raises(m.BdlmError, match="length"):
        m.bdlm_sync_status(ws)
    co.append(c, K[[3, 1]], V[[3, 1]], offsets_of([2]))
    same(cache, c)


# ---------------------------------------------------------------- together
def verify_step(m, cache, x, ws, vws):
    """One step of a one-layer target: masks, attention, probabilities, tests, commit.  Rows' keys, values and
    queries come from their tokens and positions."""
    vis, pos = m.bdlm_tree_mask(cache, x["parents"], x["off"], x["R"], workspace=ws)
    e = x["embed"][x["tokens"].long()] + x["place"][pos.long()]
    q, k, v = ((e @ x[w]).to(torch.bfloat16).reshape(len(e), h, 64) for w, h in (("wq", 4), ("wk", 2), ("wv", 2)))
    O, _ = m.bdlm_attn_tree(q, k, v, vis, cache, x["off"], x["R"], workspace=ws)
    p = torch.softmax(O.reshape(len(e), -1).float() @ x["head"], 1)
    path, acc, tok = m.bdlm_tree_verify(x["parents"], x["tokens"], p, x["draft"], x["u"], x["s"], x["off"], x["R"],
                                        workspace=vws)
    lens = m.bdlm_cache_commit(cache, k, v, path, acc, x["off"], x["R"], workspace=ws)
    return dict(path=path, acc=acc, tok=tok, lens=lens, p=p, O=O, k=k, v=v)


def step_inputs(seed, rows, V=211, kids=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    trees = [make_tree(n, kids, seed + i) for i, n in enumerate(rows)]
    T = sum(rows)
    x = dict(parents=DEV(np.concatenate(trees)), off=DEV(offsets_of(rows)), R=max(rows), embed=r(V, 96), place=r(256, 96),
             wq=r(96, 256) / 10, wk=r(96, 128) / 10, wv=r(96, 128) / 10, head=r(256, V) * 0.3,
             u=torch.rand(T, generator=g, device="cuda"), s=torch.rand(len(rows), generator=g, device="cuda"))
    x["draft"] = torch.softmax(r(T, V), 1)
    x["tokens"] = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    return x, trees


def test_a_step_of_verification(lib):
    """Its parts against the oracle on the step's own intermediate values, and the cache that it leaves
    against attention of the accepted path alone."""
    m = lib
    rows = [12, 7, 0, 20]
    c, _ = make_cache([40, 0, 9, 77], 128, 2, 64, 16, seed=1)
    cache = device_cache(m, torch, c)
    ws, vws = m.bdlm_cache_workspace(cache, 4, 20), m.bdlm_verify_workspace(4, 20, 211)
    x, trees = step_inputs(3, rows)
    y = verify_step(m, cache, x, ws, vws)
    m.bdlm_sync_status(ws)
    m.bdlm_sync_status(vws)
    off = offsets_of(rows)
    host = lambda t: t.float().cpu().numpy()
    for i in range(4):
        a, b = off[i], off[i + 1]
        want, nxt = to.verify(trees[i], host(x["tokens"])[a:b].astype(int), host(y["p"])[a:b], host(x["draft"])[a:b],
                              host(x["u"])[a:b], host(x["s"])[i], 20)
        assert y["path"][i, : len(want)].tolist() == want and y["acc"][i] == len(want) and y["tok"][i] == nxt
    lens = to.commit(c, host(y["k"]), host(y["v"]), y["path"].cpu().numpy(), y["acc"].cpu().numpy(), off)
    assert y["lens"].tolist() == lens.tolist()
    same(cache, c)


def test_a_step_is_captured_and_replayed_on_other_trees(lib):
    m = lib
    rows = [12, 7, 3, 20]
    make = lambda: device_cache(m, torch, make_cache([40, 0, 9, 77], 128, 2, 64, 16, seed=1)[0])
    cache = make()
    ws, vws = m.bdlm_cache_workspace(cache, 4, 20), m.bdlm_verify_workspace(4, 20, 211)
    x, _ = step_inputs(3, rows)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        verify_step(m, cache, x, ws, vws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = verify_step(m, cache, x, ws, vws)
        cache.lens.copy_(y["lens"])
    cache2 = make()
    for t, f in ((cache.k8, cache2.k8), (cache.v8, cache2.v8), (cache.k_scale, cache2.k_scale),
                 (cache.v_scale, cache2.v_scale), (cache.lens, cache2.lens), (cache.page_table, cache2.page_table)):
        t.copy_(f)
    for seed in (5, 6, 7):  # other trees, tokens and numbers; the cache grows from step to step
        new, _ = step_inputs(seed, rows, kids=1 + seed % 3)
        for k in ("parents", "tokens", "draft", "u", "s"):
            x[k].copy_(new[k])
        g.replay()
        z = verify_step(m, cache2, x, m.bdlm_cache_workspace(cache2, 4, 20), vws)
        cache2.lens.copy_(z["lens"])
        for k in y:
            assert torch.equal(y[k], z[k]), k
        assert torch.equal(cache.k8.view(torch.uint8), cache2.k8.view(torch.uint8)) and torch.equal(cache.lens, cache2.lens)
    m.bdlm_sync_status(ws)


def test_calls_on_another_stream(lib):
    m = lib
    rows = [12, 7, 3, 20]
    x, _ = step_inputs(4, rows)
    c, cache = small_cache(m, [40, 0, 9, 77], Hkv=2, capacity=128)
    want = m.bdlm_tree_mask(cache, x["parents"], x["off"], x["R"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = m.bdlm_tree_mask(cache, x["parents"], x["off"], x["R"], stream=st)
    p = torch.softmax(torch.randn(42, 211, device="cuda"), 1)
    a = m.bdlm_tree_verify(x["parents"], x["tokens"], p, x["draft"], x["u"], x["s"], x["off"], x["R"])
    st.wait_stream(torch.cuda.current_stream())
    b = m.bdlm_tree_verify(x["parents"], x["tokens"], p, x["draft"], x["u"], x["s"], x["off"], x["R"], stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(i, j) for i, j in zip((*want, *a), (*got, *b)))


def test_a_padded_batch_is_the_ragged_one(lib):
    """Trees of equal size, the rest of each filled with rows without a parent and any tokens, keys and values: the same
    paths, tokens, outputs and cache as packed trees with offsets."""
    m = lib
    rows, R, V, d = [5, 9, 1, 12], 12, 60, 64
    trees = [make_tree(n, 2, 3 + i) for i, n in enumerate(rows)]
    parents, tokens, target, draft, u, s = make_drafts(trees, V, 4)
    off = offsets_of(rows)
    at = np.concatenate([np.arange(R * i, R * i + n) for i, n in enumerate(rows)])
    rng = np.random.default_rng(1)

    def pad(x, fill):
        y = np.empty((4 * R,) + x.shape[1:], x.dtype)
        y[:] = fill
        y[at] = x
        return y
    P = dict(parents=pad(parents, -1), tokens=pad(tokens, 3), target=pad(target, np.nan), draft=pad(draft, np.nan),
             u=pad(u, 0.0))
    got = m.bdlm_tree_verify(*(DEV(P[k]) for k in ("parents", "tokens", "target", "draft", "u")), DEV(s))
    want = m.bdlm_tree_verify(DEV(parents), DEV(tokens), DEV(target), DEV(draft), DEV(u), DEV(s), DEV(off), R)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    Q, K, Vv = (make_rows(sum(rows), H, d, 1 + i) for i, H in enumerate((4, 2, 2)))
    make = lambda: device_cache(m, torch, make_cache([50, 0, 17, 33], 80, 2, d, 16, seed=2)[0])
    a, b = make(), make()
    va, vb = m.bdlm_tree_mask(a, DEV(P["parents"])), m.bdlm_tree_mask(b, DEV(parents), DEV(off), R)
    assert torch.equal(va[0][DEV(at)], vb[0]) and torch.equal(va[1][DEV(at)], vb[1])
    wide = [to_dev(pad(x, np.float32(np.inf)), torch) for x in (Q, K, Vv)]
    Oa, La = m.bdlm_attn_tree(*wide, va[0], a, scale=0.1)
    Ob, Lb = m.bdlm_attn_tree(*(to_dev(x, torch) for x in (Q, K, Vv)), vb[0], b, DEV(off), R, scale=0.1)
    assert torch.equal(Oa[DEV(at)], Ob) and torch.equal(La[:, DEV(at)], Lb)
    la = m.bdlm_cache_commit(a, wide[1], wide[2], got[0], got[1])
    lb = m.bdlm_cache_commit(b, *(to_dev(x, torch) for x in (K, Vv)), want[0], want[1], DEV(off), R)
    assert torch.equal(la, lb) and torch.equal(a.k8.view(torch.uint8), b.k8.view(torch.uint8))


def test_calls_side_by_side(lib):
    """Two streams, a workspace for each, the same inputs: all calls at once, many times."""
    m = lib
    rows = [12, 7, 3, 20]
    x, _ = step_inputs(4, rows)
    make = lambda: device_cache(m, torch, make_cache([200, 0, 150, 77], 240, 2, 64, 16, seed=1)[0])  # (256 places)
    a, b, c = make(), make(), make()
    wa, wb, wc = (m.bdlm_cache_workspace(y, 4, 20) for y in (a, b, c))
    va, vb, vc = (m.bdlm_verify_workspace(4, 20, 211) for _ in range(3))
    for _ in range(10):  # (a commit may round the old codes of its first block to a larger scale: once)
        want = verify_step(m, c, x, wc, vc)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(sa):
            ya = verify_step(m, a, x, wa, va)
        with torch.cuda.stream(sb):
            yb = verify_step(m, b, x, wb, vb)
    torch.cuda.synchronize()
    for k in ("path", "acc", "tok", "lens", "O"):
        assert torch.equal(ya[k], want[k]) and torch.equal(yb[k], want[k]), k
    for w in (wa, wb, va, vb):
        m.bdlm_sync_status(w)


def test_verify_repeats_bitwise_in_any_company(lib):
    """A sequence's result does not depend on how many others there are (other clusters, other runs of the
    vocabulary)."""
    m = lib
    trees = [make_tree(16, 3, 1)]
    parents, tokens, target, draft, u, s = make_drafts(trees, 5003, 2)
    one = m.bdlm_tree_verify(DEV(parents), DEV(tokens), DEV(target), DEV(draft), DEV(u), DEV(s))
    for n in (2, 90, 200, 700):
        t = lambda x: DEV(np.concatenate([x] * n))
        many = m.bdlm_tree_verify(t(parents), t(tokens), t(target), t(draft), t(u), t(s))
        for a, b in zip(one, many):
            assert (b == a).all()


def test_no_rows_at_all(lib):
    m = lib
    c, cache = small_cache(m, [20, 3], capacity=32)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    vis, pos = m.bdlm_tree_mask(cache, none, off, 1)
    assert vis.shape == (0, 1) and pos.shape == (0,)
    Q, K = to_dev(make_rows(0, 2, 64, 1), torch), to_dev(make_rows(0, 1, 64, 1), torch)
    O, LSE = m.bdlm_attn_tree(Q, K, K, vis, cache, off)
    assert O.shape == (0, 2, 64) and LSE.shape == (2, 0)
    p = torch.zeros((0, 9), device="cuda")
    path, acc, tok = m.bdlm_tree_verify(none, none, p, p, p[:, 0].contiguous(), torch.rand(2, device="cuda"), off, 1)
    assert path.tolist() == [[-1], [-1]] and acc.tolist() == [0, 0] and tok.tolist() == [-1, -1]
    assert m.bdlm_cache_commit(cache, K, K, path, acc, off).tolist() == [20, 3]
    same(cache, c)
