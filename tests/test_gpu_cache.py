"""The 8-bit cache's calls on the GPU against the fp64 oracle.

Tolerances, from the arithmetic (eps / 2 of a type is its largest rounding):
  * codes, scales, lengths, kept positions: equal;
  * O: p_ij is rounded to bf16 at worst (2^-8; in parts for an fp32 O,
    2^-22), V's codes and scales are exact, so |dO| <= (2^-8 or 2^-22, + c)
    sum_j p_ij |v_j|, plus 2^-8 |O| when O is bf16; c covers the fp32 scores
    (next line) and the exponential, twice (p and the row sum);
  * a score is an fp32 sum of d products: off by at most (d + 8) 2^-24 times
    scale sum |q k|, whose largest value in the row is the oracle's E; the
    exponent x log2(e) and exp2 add 2^-22 each, and |LSE| its own rounding.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle.cache_oracle as co
from structured_mask_attention_gb300.inputs import bf16_round
from tests.cache_util import device_cache, host_codes, make_cache, make_rows, offsets_of
from tests.parity_util import to_dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8  # bf16's largest rounding


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import structured_mask_attention_gb300 as m
    m.load_library()
    return m


def score_error(d, E):
    return (d + 8) * 2.0 ** -24 * E + 2.0 ** -21


def check_attn(O, LSE, ref, d, bf16_out):
    Or, Lr, A, E = ref
    O, LSE = O.double().cpu().numpy(), LSE.double().cpu().numpy()
    live = np.isfinite(Lr)
    assert (np.isneginf(LSE) == ~live).all() and np.isfinite(O).all()
    ds = score_error(d, E)
    tol = ((HALF if bf16_out else 2.0 ** -22) + 2 * ds.T[:, :, None]) * A + (HALF * np.abs(Or) if bf16_out else 0) + 1e-30
    worst = (np.abs(O - Or) / tol).max()
    lerr = (np.abs(LSE[live] - Lr[live]) / (ds[live] + 2.0 ** -22 * (1 + np.abs(Lr[live])))).max() if live.any() else 0.0
    print(f"  O {worst:.3f} of its tolerance, LSE {lerr:.3f}")
    assert worst <= 1 and lerr <= 1
    assert (O[~live.T] == 0).all()


def run_attn(m, lens, rows, Hq, Hkv, d, page, local=True, o_dtype=None, seed=0, uniform=False, extra=0, capacity=None):
    c, _ = make_cache(lens, capacity or max(max(lens), 1), Hkv, d, page, seed)
    off, T = offsets_of(rows), int(sum(rows)) + extra
    Q, K, V = (make_rows(T, H, d, seed + i + 1) for i, H in enumerate((Hq, Hkv, Hkv)))
    cache = device_cache(m, torch, c)
    ws = m.bdlm_cache_workspace(cache, Hq, max(rows))
    out = (torch.full((T, Hq, d), 7.0, dtype=o_dtype or torch.bfloat16, device="cuda"),
           torch.full((Hq, T), 7.0, dtype=torch.float32, device="cuda"))
    kv = (to_dev(K, torch), to_dev(V, torch)) if local else (None, None)
    doff = None if uniform else torch.from_numpy(off).cuda()
    m.bdlm_attn_cached(to_dev(Q, torch), *kv, cache, doff, max(rows), out=out, workspace=ws)
    m.bdlm_sync_status(ws)
    n = int(off[-1])
    ref = co.attn(c, Q[:n], K[:n] if local else None, V[:n], off, 1 / math.sqrt(d))
    check_attn(out[0][:n], out[1][:, :n], ref, d, out[0].dtype == torch.bfloat16)
    assert (out[0][n:] == 7).all() and (out[1][:, n:] == 7).all(), "rows behind the last sequence were touched"


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_attn_single_tokens(lib, page, d):
    """One token each: lengths around pages and units, 0 and 1 among them."""
    run_attn(lib, [0, 1, 15, 16, 17, 127, 128, 129, 300, 33], [1] * 10, 8, 2, d, page, seed=page + d)


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (16, 8), (10, 2), (16, 1), (17, 1), (40, 1)])
def test_attn_head_groups(lib, Hq, Hkv):
    run_attn(lib, [200, 77], [1, 2], Hq, Hkv, 64, 16, seed=Hq)


@pytest.mark.parametrize("rows", [[3, 1, 0, 5], [32, 31, 33, 1], [128, 100, 129, 7], [300, 257, 64, 0]])
@pytest.mark.parametrize("local", [True, False])
def test_attn_blocks(lib, rows, local):
    run_attn(lib, [260, 0, 128, 411], rows, 4, 2, 64, 32, local=local, seed=sum(rows), extra=3)


@pytest.mark.parametrize("rows", [[16, 9], [65, 64], [200, 130]])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
def test_attn_blocks_d128(lib, rows, o_dtype):
    run_attn(lib, [700, 391], rows, 6, 2, 128, 64, o_dtype=o_dtype, seed=sum(rows))


def test_attn_uniform_rows_without_offsets(lib):
    run_attn(lib, [50, 90, 0], [8, 8, 8], 4, 2, 64, 16, uniform=True, seed=5)


@pytest.mark.parametrize("rows", [1, 40])
def test_attn_long_prefix_spans_many_parts(lib, rows):
    run_attn(lib, [6000, 1], [rows, 1], 4, 1, 64, 128, seed=9)


@pytest.mark.parametrize("rows,chain", [(1, 2), (10, 2), (40, 32), (150, 32)])
def test_attn_fp32_output_of_long_rows(lib, rows, chain):
    """Sequences of many keys of like weight (the same pages, other queries),
    so that a CTA adds up tens of key tiles.  The tensor cores cut each sum
    off by up to 2^-23 of it, always towards zero; ``chain`` products of 16 keys
    follow each other before the threads take over with rounded sums.  A sum of
    terms unlike in sign grows as the root of their number, 2/3 of its last size
    in the mean: off by chain * 2^-23 * 2/3 at most, here 2^-22.6 or 2^-18.6 of O.
    The weights' and scores' own errors, 2^-22 a few times over, are unlike in
    sign from key to key: 2^-21 of O in the mean."""
    m = lib
    d, n, L = 128, 24, 12000
    c, _ = make_cache([L], L, 2, d, 64, seed=93)
    c["table"], c["lens"] = np.repeat(c["table"], n, 0), np.repeat(c["lens"], n)
    Q = make_rows(n * rows, 4, d, 3)
    O, LSE = m.bdlm_attn_cached(to_dev(Q, torch), None, None, device_cache(m, torch, c), o_dtype=torch.float32)
    ref = co.attn(c, Q, None, None, offsets_of([rows] * n), 1 / math.sqrt(d))
    check_attn(O, LSE, ref, d, False)
    diff = O.double().cpu().numpy() - ref[0]
    rel = math.sqrt((diff ** 2).sum() / (ref[0] ** 2).sum())
    print(f"  O off by {rel:.2e} of its size")
    assert rel <= chain * 2.0 ** -23 * 2 / 3 + 2.0 ** -21


def test_attn_many_sequences(lib):
    lens = [(37 * i) % 200 for i in range(70)]
    run_attn(lib, lens, [1 + i % 3 for i in range(70)], 4, 2, 64, 16, seed=11)


def test_attn_scales_of_unlike_pages(lib):
    """Blocks whose scales differ by 2^40: each weighs in at its own scale."""
    m = lib
    c, _ = make_cache([96], 96, 1, 64, 16, seed=13)
    c["vs"][c["table"][0, 1]] = 2.0 ** 30
    c["vs"][c["table"][0, 3]] = 2.0 ** -50
    c["ks"][c["table"][0, 4]] = 2.0 ** -60
    Q = make_rows(2, 2, 64, 1)
    cache = device_cache(m, torch, c)
    O, LSE = m.bdlm_attn_cached(to_dev(Q, torch), None, None, cache, None, 2, o_dtype=torch.float32)
    check_attn(O, LSE, co.attn(c, Q, None, None, offsets_of([2]), 0.125), 64, False)


@pytest.mark.parametrize("factor", [2.0 ** -100, 2.0 ** 60, 40.0])
def test_attn_queries_of_any_size(lib, factor):
    m = lib
    c, _ = make_cache([150], 150, 1, 64, 32, seed=17)
    for rows in (1, 24):
        Q = bf16_round(make_rows(rows, 2, 64, 1) * np.float32(factor))  # the oracle reads what the device holds
        sc = 0.125 / factor if factor > 1e3 else 0.125
        cache = device_cache(m, torch, c)
        O, LSE = m.bdlm_attn_cached(to_dev(Q, torch), None, None, cache, None, rows, scale=sc, o_dtype=torch.float32)
        check_attn(O, LSE, co.attn(c, Q, None, None, offsets_of([rows]), sc), 64, False)


@pytest.mark.parametrize("rows", [1, 50])
def test_attn_nan_scale_poisons_the_rows_that_see_it_only(lib, rows):
    m = lib
    c, _ = make_cache([40, 40], 48, 1, 64, 16, seed=19)
    c["vs"][c["table"][0, 1]] = np.nan
    Q = make_rows(2 * rows, 2, 64, 1)
    cache = device_cache(m, torch, c)
    O, LSE = m.bdlm_attn_cached(to_dev(Q, torch), None, None, cache, None, rows)
    assert torch.isnan(O[:rows]).all() and torch.isfinite(O[rows:]).all() and torch.isfinite(LSE[:, rows:]).all()


@pytest.mark.parametrize("rows", [[1, 1, 1], [7, 3, 9], [40, 3, 70], [130, 200, 5]])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_attn_other_rows_stay_out(lib, rows, value):
    """Whatever the rows of another sequence, or those behind the last one,
    hold: a sequence's result does not know of them."""
    m = lib
    d, Hq, Hkv = 64, 4, 2
    c, _ = make_cache([150, 20, 0], 150, Hkv, d, 16, seed=sum(rows))
    off, T = offsets_of(rows), sum(rows) + 9
    Q, K, V = (make_rows(T, H, d, 1 + i) for i, H in enumerate((Hq, Hkv, Hkv)))
    ref = co.attn(c, Q[:T - 9], K[:T - 9], V[:T - 9], off, 0.125)
    mine = np.r_[0:off[1], off[2]:off[3]]
    for x in (Q, K, V):
        x[off[1]:off[2]] = value
        x[off[3]:] = value
    cache = device_cache(m, torch, c)
    O, LSE = m.bdlm_attn_cached(*(to_dev(x, torch) for x in (Q, K, V)), cache, torch.from_numpy(off).cuda(), max(rows),
                                o_dtype=torch.float32)
    check_attn(O[mine], LSE[:, mine], (ref[0][mine], ref[1][:, mine], ref[2][mine], ref[3][:, mine]), d, False)
    W = torch.zeros((3, Hkv, c["table"].shape[1] * 16), device="cuda")
    m.bdlm_cache_weights(to_dev(Q, torch), LSE, cache, W, torch.from_numpy(off).cuda(), max(rows))
    assert torch.isfinite(W[0]).all() and (W[2] == 0).all()


@pytest.mark.parametrize("rows", [2, 30, 70, 140])
def test_attn_query_row_that_is_not_finite(lib, rows):
    m = lib
    c, _ = make_cache([200], 200, 1, 128, 32, seed=29)
    Q = make_rows(rows, 2, 128, 1)
    ref = co.attn(c, Q, None, None, offsets_of([rows]), 0.125)
    Q[1, 0, 5], Q[1, 1, 9] = math.inf, math.nan
    O, LSE = m.bdlm_attn_cached(to_dev(Q, torch), None, None, device_cache(m, torch, c), scale=0.125,
                                o_dtype=torch.float32)
    mine = np.r_[0:1, 2:rows]
    assert torch.isnan(O[1]).all()
    check_attn(O[mine], LSE[:, mine], (ref[0][mine], ref[1][:, mine], ref[2][mine], ref[3][:, mine]), 128, False)


@pytest.mark.parametrize("rows", [[90, 60], [400, 300]])
@pytest.mark.parametrize("page,d", [(16, 128), (128, 64), (32, 128)])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
def test_attn_tiles_by_page(lib, rows, page, d, o_dtype):
    run_attn(lib, [777, 1290], rows, 2, 1, d, page, o_dtype=o_dtype, seed=page + d, extra=1)


@pytest.mark.parametrize("rows", [40, 150])
def test_attn_blocks_of_many_sequences(lib, rows):
    run_attn(lib, [(53 * i) % 300 for i in range(40)], [rows - i % 3 for i in range(40)], 2, 1, 64, 32, seed=rows)


def test_no_rows_at_all(lib):
    m = lib
    c, _ = make_cache([20, 3], 32, 1, 64, 16, seed=37)
    cache, off = device_cache(m, torch, c), torch.zeros(3, dtype=torch.int32, device="cuda")
    Q, K = to_dev(make_rows(0, 2, 64, 1), torch), to_dev(make_rows(0, 1, 64, 1), torch)
    O, LSE = m.bdlm_attn_cached(Q, K, K, cache, off)
    assert O.shape == (0, 2, 64) and LSE.shape == (2, 0)
    W = torch.ones((2, 1, 32), device="cuda")
    m.bdlm_cache_weights(Q, LSE, cache, W, off)
    assert (W == 1).all()
    assert m.bdlm_cache_append(cache, K, K, off).tolist() == [20, 3]
    same_cache(cache, c)


def test_attn_repeats_bitwise(lib):
    m = lib
    c, _ = make_cache([3000, 17, 900], 3000, 2, 128, 64, seed=23)
    cache = device_cache(m, torch, c)
    for rows in (1, 48):
        Q = to_dev(make_rows(3 * rows, 8, 128, 2), torch)
        a = m.bdlm_attn_cached(Q, None, None, cache, None, rows, o_dtype=torch.float32)
        b = m.bdlm_attn_cached(Q, None, None, cache, None, rows, o_dtype=torch.float32)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [[1, 1, 1, 1, 1], [5, 0, 40, 17, 129], [300, 1, 2, 3, 64]])
def test_append(lib, page, d, rows):
    m = lib
    lens = [0, 3, page - 1, page, 2 * page + 5]
    c, _ = make_cache(lens, max(lens) + max(rows), 3, d, page, seed=sum(rows) + page)
    off, T = offsets_of(rows), sum(rows)
    grow = np.exp(np.random.default_rng(3).uniform(-6, 6, (T, 1, 1))).astype(np.float32)  # old blocks get new scales
    K, V = (bf16_round(make_rows(T, 3, d, s) * grow) for s in (1, 2))
    K[T // 2] = 0.0
    cache = device_cache(m, torch, c)
    ws = m.bdlm_cache_workspace(cache)
    got = m.bdlm_cache_append(cache, to_dev(K, torch), to_dev(V, torch), torch.from_numpy(off).cuda(), max(rows),
                              workspace=ws)
    m.bdlm_sync_status(ws)
    want = co.append(c, K, V, off)
    assert got.cpu().tolist() == want.tolist() and cache.lens.cpu().tolist() == lens
    same_cache(cache, c)


def same_cache(cache, c):
    for w in ("k", "v"):
        assert np.array_equal(host_codes(getattr(cache, w + "8")), c[w + "8"])
        assert np.array_equal(getattr(cache, w + "_scale").cpu().numpy(), c[w + "s"], equal_nan=True)


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_append_of_a_value_that_is_not_finite(lib, value):
    """Its block (old tokens too) reads NaN, its neighbours do not."""
    m = lib
    c, _ = make_cache([3], 64, 2, 64, 16, seed=31)
    K = make_rows(30, 2, 64, 1)
    K[4, 1, 7] = value
    cache = device_cache(m, torch, c)
    m.bdlm_cache_append(cache, to_dev(K, torch), to_dev(K, torch))
    s = cache.k_scale.cpu().numpy()[c["table"][0, :3]]
    assert np.isnan(s[0, 1]) and np.isfinite(np.delete(s.ravel(), 1)).all()


def test_append_behind_a_scale_that_is_no_power_of_two(lib):
    m = lib
    c, _ = make_cache([7, 7], 32, 1, 64, 16, seed=33)
    c["ks"][c["table"][0, 0]] = 0.037
    c["ks"][c["table"][1, 0]] = 7.3
    K = make_rows(2, 1, 64, 1)
    cache = device_cache(m, torch, c)
    m.bdlm_cache_append(cache, to_dev(K, torch), to_dev(K, torch))
    co.append({**c, "ks": c["ks"], "vs": c["vs"]}, K, K, offsets_of([1, 1]))
    assert np.array_equal(cache.k_scale.cpu().numpy(), c["ks"], equal_nan=True)
    assert np.array_equal(host_codes(cache.k8), c["k8"])


# ----------------------------------------------------------------- weights
@pytest.mark.parametrize("lens,rows,Hq,Hkv,d,page", [
    ([0, 1, 127, 128, 300], [1, 1, 1, 1, 1], 8, 2, 128, 64),
    ([100, 33, 260], [40, 0, 129], 6, 2, 64, 16),
    ([513], [300], 2, 1, 64, 128),
    ([200, 200], [17, 64], 5, 1, 128, 32),
    ([700], [70], 40, 4, 64, 64),
])
def test_weights(lib, lens, rows, Hq, Hkv, d, page):
    m = lib
    c, _ = make_cache(lens, max(lens) + 5, Hkv, d, page, seed=sum(lens))
    off, T = offsets_of(rows), sum(rows)
    Q = make_rows(T, Hq, d, 3)
    LSE = co.attn(c, Q, None, None, off, 1 / math.sqrt(d))[1].astype(np.float32)
    cap = c["table"].shape[1] * page
    W0 = np.random.default_rng(5).random((len(lens), Hkv, cap), dtype=np.float32)
    cache = device_cache(m, torch, c)
    ws = m.bdlm_cache_workspace(cache)
    W = torch.from_numpy(W0.copy()).cuda()
    for _ in range(2):  # adds
        m.bdlm_cache_weights(to_dev(Q, torch), torch.from_numpy(LSE).cuda(), cache, W, torch.from_numpy(off).cuda(),
                             max(max(rows), 1), workspace=ws)
    m.bdlm_sync_status(ws)
    once, E = co.weights(c, Q, LSE, off, 1 / math.sqrt(d), np.zeros_like(W0))
    ref = W0 + 2 * once
    # each p: its score's error and the rounding of LSE log2(e) (2^-24 of it); sums of n terms in fp32
    n = max(rows) * (Hq // Hkv) + 4
    rel = score_error(d, E) + 2.0 ** -23 * (1 + np.abs(LSE[np.isfinite(LSE)]).max()) + n * 2.0 ** -24
    err = np.abs(W.double().cpu().numpy() - ref)
    print(f"  weights {(err / (rel * ref + 2.0 ** -24)).max():.3f} of its tolerance")
    assert (err <= rel * ref + 2.0 ** -24).all()
    for s, L in enumerate(lens):
        assert np.array_equal(W[s, :, L:].cpu().numpy(), W0[s, :, L:])


@pytest.mark.parametrize("lens,rows,Hq,Hkv,d,page", [
    ([4800, 3000], [384, 384], 16, 8, 128, 64),        # three chunks of 256 rows, three key tiles per CTA
    ([9000, 2000, 5000], [330, 260, 384], 4, 2, 64, 16),
    ([9000, 20000], [200, 90], 40, 2, 128, 128),       # 16 and 8 chunks
])
def test_weights_of_several_chunks_and_tiles(lib, lens, rows, Hq, Hkv, d, page):
    """A CTA goes through several chunks of rows and several segments: each
    time with its own rows' constants, whichever sub-tile is ahead."""
    m = lib
    c, _ = make_cache(lens, max(lens), Hkv, d, page, seed=sum(rows))
    off, T = offsets_of(rows), sum(rows)
    Q = make_rows(T, Hq, d, 3)
    dQ, doff, cache = to_dev(Q, torch), torch.from_numpy(off).cuda(), device_cache(m, torch, c)
    ws = m.bdlm_cache_workspace(cache, Hq, max(rows))
    LSE = m.bdlm_attn_cached(dQ, None, None, cache, doff, max(rows), workspace=ws, o_dtype=torch.float32)[1]
    def once():
        W = torch.zeros((len(lens), Hkv, c["table"].shape[1] * page), device="cuda")
        return m.bdlm_cache_weights(dQ, LSE, cache, W, doff, max(rows), workspace=ws)
    W = once()
    for _ in range(50):
        assert torch.equal(once(), W)
    m.bdlm_sync_status(ws)
    L = LSE.cpu().numpy()
    ref, E = co.weights(c, Q, L, off, 1 / math.sqrt(d), np.zeros(W.shape, np.float32))
    rel = score_error(d, E) + 2.0 ** -23 * (1 + np.abs(L).max()) + (max(rows) * (Hq // Hkv) + 4) * 2.0 ** -24
    assert (np.abs(W.double().cpu().numpy() - ref) <= rel * ref + 2.0 ** -24).all()


def test_weights_of_rows_without_a_key(lib):
    """LSE = -inf rows (a block whose other keys were not given) add nothing."""
    m = lib
    c, _ = make_cache([20], 32, 1, 64, 16, seed=41)
    Q = make_rows(3, 2, 64, 1)
    LSE = torch.full((2, 3), -math.inf, device="cuda")
    W = torch.zeros((1, 1, 32), device="cuda")
    m.bdlm_cache_weights(to_dev(Q, torch), LSE, device_cache(m, torch, c), W)
    assert (W == 0).all()


# ------------------------------------------------------------------- evict
@pytest.mark.parametrize("lens,keep,sinks,recent,page,d", [
    ([100, 20, 0, 64], 32, 4, 8, 16, 64),
    ([100, 20, 33, 64], 33, 0, 0, 32, 128),
    ([500, 1], 200, 200, 0, 64, 64),
    ([500, 130], 129, 0, 129, 128, 128),
    ([3000, 2049], 1, 0, 0, 16, 64),
    ([3000, 2049], 2500, 100, 1000, 64, 64),
    ([90, 80], 1000, 4, 8, 16, 64),  # nothing to evict: the tokens move
])
@pytest.mark.parametrize("kind", ["random", "ties", "signed"])
def test_evict(lib, lens, keep, sinks, recent, page, d, kind):
    m = lib
    Hkv = 2
    c, (dst,) = make_cache(lens, max(lens) + 3, Hkv, d, page, seed=keep + sum(lens), sets=2)
    cap = c["table"].shape[1] * page
    rng = np.random.default_rng(keep)
    W = rng.random((len(lens), Hkv, cap), dtype=np.float32)
    if kind == "ties":
        W = (W * 3).astype(np.int32).astype(np.float32)
        W[W == 1] = -0.0
    elif kind == "signed":
        W = (W - 0.5) * np.exp(rng.uniform(-60, 60, W.shape)).astype(np.float32)
        W[..., 5:7] = np.nan
    cache = device_cache(m, torch, c)
    ws = m.bdlm_cache_workspace(cache, keep=keep)
    kept = torch.full((len(lens), Hkv, keep), 9, dtype=torch.int32, device="cuda")
    lo, wo, _ = m.bdlm_cache_evict(cache, torch.from_numpy(W).cuda(), torch.from_numpy(dst).cuda(), keep, sinks,
                                   recent, kept=kept, workspace=ws)
    m.bdlm_sync_status(ws)
    rl, rw, rk = co.evict(c, W, dst, keep, sinks, recent)
    assert np.array_equal(kept.cpu().numpy(), rk)
    assert np.array_equal(lo.cpu().numpy(), rl)
    assert np.array_equal(wo.cpu().numpy(), rw, equal_nan=True)
    same_cache(cache, c)


@pytest.mark.parametrize("lens,capacity,page,keep", [
    ([30000, 9000], 33000, 64, 10000),       # clusters of CTAs
    ([361000], 400000, 128, 200001),         # runs longer than a CTA holds
    ([50] * 90, 64, 16, 20),                 # more selections than SMs
])
def test_evict_long_and_many(lib, lens, capacity, page, keep):
    m = lib
    c, (dst,) = make_cache(lens, capacity, 1, 64, page, seed=keep, sets=2)
    cap = c["table"].shape[1] * page
    W = np.random.default_rng(1).random((len(lens), 1, cap), dtype=np.float32) ** 8
    W[:, :, ::5] = 0.25  # a tie around the cut
    cache = device_cache(m, torch, c)
    ws = m.bdlm_cache_workspace(cache)
    lo, wo, kept = m.bdlm_cache_evict(cache, torch.from_numpy(W).cuda(), torch.from_numpy(dst).cuda(), keep, 3, 7,
                                      workspace=ws)
    m.bdlm_sync_status(ws)
    rl, rw, rk = co.evict(c, W, dst, keep, 3, 7)
    assert np.array_equal(kept.cpu().numpy(), rk) and lo.cpu().tolist() == rl.tolist()
    assert np.array_equal(wo.cpu().numpy(), rw)
    same_cache(cache, c)


@pytest.mark.parametrize("rows", [1, 60])
def test_weights_of_many_sequences(lib, rows):
    m = lib
    n = 45
    c, _ = make_cache([(31 * i) % 280 for i in range(n)], 280, 2, 64, 16, seed=43)
    off, T = offsets_of([rows] * n), n * rows
    Q = make_rows(T, 4, 64, 3)
    LSE = co.attn(c, Q, None, None, off, 0.125)[1].astype(np.float32)
    W = torch.zeros((n, 2, c["table"].shape[1] * 16), device="cuda")
    m.bdlm_cache_weights(to_dev(Q, torch), torch.from_numpy(LSE).cuda(), device_cache(m, torch, c), W)
    ref, E = co.weights(c, Q, LSE, off, 0.125, np.zeros(W.shape, np.float32))
    rel = score_error(64, E) + 2.0 ** -23 * (1 + np.abs(LSE[np.isfinite(LSE)]).max()) + (2 * rows + 4) * 2.0 ** -24
    assert (np.abs(W.double().cpu().numpy() - ref) <= rel * ref + 2.0 ** -24).all()


@pytest.mark.parametrize("rows", [1, 48, 150])
def test_pool_past_32_bits(lib, rows):
    """Pages at the end of a pool of 4.6 GB of codes: every call's offsets."""
    m = lib
    Hkv, d, page = 2, 128, 64
    c, (dst,) = make_cache([300, 129], 700, Hkv, d, page, seed=91, sets=2)
    n, n_pages = c["k8"].shape[0], 280_000
    assert (n_pages - n) * Hkv * page * d > 2 ** 32 and n_pages * Hkv * page * d * 2 < 20e9
    shift = n_pages - n
    pool = [torch.empty((n_pages, Hkv, page, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.empty((n_pages, Hkv), device="cuda") for _ in range(2)]
    for w, p, s in zip("kv", pool, sc):
        p[shift:] = torch.from_numpy(c[w + "8"]).cuda()
        s[shift:] = torch.from_numpy(c[w + "s"]).cuda()
    dev = lambda t: torch.from_numpy(t + np.int32(shift)).cuda()
    cache = m.BdlmCache(*(p.view(torch.float8_e4m3fn) for p in pool), *sc, dev(c["table"]),
                        torch.from_numpy(c["lens"]).cuda())
    off = offsets_of([rows, rows])
    Q, K, V = (make_rows(2 * rows, H, d, 1 + i) for i, H in enumerate((4, Hkv, Hkv)))
    dq, dk, dv = (to_dev(x, torch) for x in (Q, K, V))
    ws = m.bdlm_cache_workspace(cache, 4, rows, 200)
    O, LSE = m.bdlm_attn_cached(dq, dk, dv, cache, workspace=ws)
    check_attn(O, LSE, co.attn(c, Q, K, V, off, 1 / math.sqrt(d)), d, True)
    W = torch.zeros((2, Hkv, c["table"].shape[1] * page), device="cuda")
    m.bdlm_cache_weights(dq, LSE, cache, W, workspace=ws)
    ref, E = co.weights(c, Q, LSE.cpu().numpy(), off, 1 / math.sqrt(d), np.zeros(W.shape, np.float32))
    rel = score_error(d, E) + 2.0 ** -23 * (1 + LSE.abs().max().item()) + (2 * rows + 4) * 2.0 ** -24
    assert (np.abs(W.double().cpu().numpy() - ref) <= rel * ref + 2.0 ** -24).all()
    cache.lens.copy_(m.bdlm_cache_append(cache, dk, dv, workspace=ws))
    c["lens"] = co.append(c, K, V, off)
    lo, wo, kept = m.bdlm_cache_evict(cache, W, dev(dst), 200, 4, 8, workspace=ws)
    m.bdlm_sync_status(ws)
    rl, rw, rk = co.evict(c, W.cpu().numpy(), dst, 200, 4, 8)
    assert np.array_equal(kept.cpu().numpy(), rk) and lo.cpu().tolist() == rl.tolist()
    assert np.array_equal(wo.cpu().numpy(), rw)
    for w, p, s in zip("kv", pool, sc):
        assert np.array_equal(p[shift:].cpu().numpy(), c[w + "8"])
        assert np.array_equal(s[shift:].cpu().numpy(), c[w + "s"], equal_nan=True)


def test_two_streams_with_a_workspace_each(lib):
    m = lib
    c, _ = make_cache([5000, 30], 5000, 2, 64, 64, seed=87)
    cache = device_cache(m, torch, c)
    Qs = [to_dev(make_rows(2 * r, 8, 64, r), torch) for r in (1, 48)]
    ref = [m.bdlm_attn_cached(q, None, None, cache) for q in Qs]
    ws = [m.bdlm_cache_workspace(cache, 8, r) for r in (1, 48)]
    out = [tuple(torch.empty_like(t) for t in r) for r in ref]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Qs]
    for _ in range(20):
        for q, w, o, st in zip(Qs, ws, out, streams):
            m.bdlm_attn_cached(q, None, None, cache, out=o, workspace=w, stream=st)
    torch.cuda.synchronize()
    for o, r in zip(out, ref):
        assert torch.equal(o[0], r[0]) and torch.equal(o[1], r[1])


# -------------------------------------------------------- contents out of range
@pytest.mark.parametrize("rows", [1, 20])
def test_contents_out_of_range_are_left_out_and_reported(lib, rows):
    """Page ids outside the pool, lengths outside the table, row offsets that
    leave the rows: the kernels check each before any access."""
    m = lib
    def fresh():
        c, (dst,) = make_cache([60, 60], 64, 1, 64, 16, seed=51, sets=2)
        return c, dst, device_cache(m, torch, c)
    Q, K = make_rows(2 * rows, 2, 64, 1), make_rows(2 * rows, 1, 64, 2)
    off = offsets_of([rows, rows])
    dQ, dK = to_dev(Q, torch), to_dev(K, torch)
    calls = {
        "attn": lambda ca, ws, o: m.bdlm_attn_cached(dQ, None, None, ca, o, rows, workspace=ws, o_dtype=torch.float32),
        "weights": lambda ca, ws, o: m.bdlm_cache_weights(dQ, torch.zeros((2, 2 * rows), device="cuda"), ca,
                                                          torch.zeros((2, 1, 64), device="cuda"), o, rows, workspace=ws),
        "append": lambda ca, ws, o: m.bdlm_cache_append(ca, dK, dK, o, rows, workspace=ws)}
    for name, call in calls.items():
        for what, msg in (("page", "page id"), ("len", "length"), ("rows", "row offsets")):
            c, dst, cache = fresh()
            ws, o = m.bdlm_cache_workspace(cache, 2, rows, 16), torch.from_numpy(off).cuda()
            if what == "page":
                cache.page_table[0, 3] = [1 << 30, -5][rows > 1]
            elif what == "len":
                cache.lens[0] = [-3, 1000][rows > 1]
                if name == "append":
                    cache.lens[0] = 1000  # no room: nothing is written for it
            else:
                o[1] = -7
            out = call(cache, ws, o)
            with pytest.raises(m.BdlmError, match=msg):
                m.bdlm_sync_status(ws)
            m.bdlm_sync_status(ws)  # read once
            if name == "attn" and what == "page":  # the page's keys are unseen
                c["lens"] = np.array([48, 60], np.int32)
                check_attn(*out, co.attn(c, Q, None, None, off, 0.125), 64, False)
    c, dst, cache = fresh()
    bad = torch.from_numpy(dst).cuda()
    bad[1, 0] = 10 ** 9
    ws = m.bdlm_cache_workspace(cache, keep=16)
    m.bdlm_cache_evict(cache, torch.rand((2, 1, 64), device="cuda"), bad, 16, workspace=ws)
    with pytest.raises(m.BdlmError, match="page id"):
        m.bdlm_sync_status(ws)


@pytest.mark.parametrize("what", ["len", "rows"])
@pytest.mark.parametrize("rows", [1, 20, 48, 150])
@pytest.mark.parametrize("n,at", [(3, 2), (40, 0), (40, 37)])
def test_whichever_sequence_is_out_of_range_is_reported(lib, what, rows, n, at):
    m = lib
    c, _ = make_cache([40] * n, 48, 1, 64, 16, seed=53)
    dQ, dK = (to_dev(make_rows(n * rows, H, 64, H), torch) for H in (2, 1))
    for name in ("attn", "weights", "append"):
        cache = device_cache(m, torch, c)
        ws, o = m.bdlm_cache_workspace(cache, 2, rows), torch.from_numpy(offsets_of([rows] * n)).cuda()
        if what == "len":
            cache.lens[at] = 1000
        else:
            o[at + 1] = n * rows + 5
        if name == "attn":
            m.bdlm_attn_cached(dQ, None, None, cache, o, rows, workspace=ws)
        elif name == "weights":
            m.bdlm_cache_weights(dQ, torch.zeros((2, n * rows), device="cuda"), cache,
                                 torch.zeros((n, 1, 48), device="cuda"), o, rows, workspace=ws)
        else:
            m.bdlm_cache_append(cache, dK, dK, o, rows, workspace=ws)
        with pytest.raises(m.BdlmError, match="length|row offsets"):
            m.bdlm_sync_status(ws)


# ------------------------------------------------------------ as they are used
def decode(m, c, dst, blocks, B, Hq, Hkv, d, keep, step):
    """Blocks of B tokens, one after the other: attend, append, weigh; then evict."""
    for b in range(blocks):
        step(b, make_rows(2 * B, Hq, d, 3 * b), make_rows(2 * B, Hkv, d, 3 * b + 1), make_rows(2 * B, Hkv, d, 3 * b + 2))


@pytest.mark.parametrize("B,d,page", [(1, 64, 16), (24, 128, 32)])
def test_decode_loop_against_the_oracle(lib, B, d, page):
    m = lib
    Hq, Hkv, keep, blocks = 8, 2, 48, 4
    c, (dst,) = make_cache([70, 0], 70 + blocks * B + B, Hkv, d, page, seed=61, sets=2)
    cap = c["table"].shape[1] * page
    W = np.zeros((2, Hkv, cap), np.float32)
    cache, dW = device_cache(m, torch, c), torch.zeros((2, Hkv, cap), device="cuda")
    ws, off = m.bdlm_cache_workspace(cache, Hq, B, keep), offsets_of([B, B])
    sc = 1 / math.sqrt(d)

    def step(b, Q, K, V):
        nonlocal W
        dq, dk, dv = (to_dev(x, torch) for x in (Q, K, V))
        O, LSE = m.bdlm_attn_cached(dq, dk, dv, cache, workspace=ws)
        check_attn(O, LSE, co.attn(c, Q, K, V, off, sc), d, True)
        m.bdlm_cache_weights(dq, LSE, cache, dW, workspace=ws)
        W, E = co.weights(c, Q, LSE.cpu().numpy(), off, sc, W)
        assert np.allclose(dW.cpu().numpy(), W, rtol=1e-4, atol=1e-6)
        cache.lens.copy_(m.bdlm_cache_append(cache, dk, dv, workspace=ws))
        c["lens"] = co.append(c, K, V, off)
        same_cache(cache, c)

    decode(m, c, dst, blocks, B, Hq, Hkv, d, keep, step)
    W32 = dW.cpu().numpy()
    lo, wo, kept = m.bdlm_cache_evict(cache, dW, torch.from_numpy(dst).cuda(), keep, 2, 8, workspace=ws)
    rl, rw, rk = co.evict(c, W32, dst, keep, 2, 8)
    assert np.array_equal(kept.cpu().numpy(), rk) and np.array_equal(wo.cpu().numpy(), rw)
    same_cache(cache, c)
    c["table"], c["lens"], W = dst, rl, rw
    cache.page_table.copy_(torch.from_numpy(dst))
    cache.lens.copy_(lo)
    dW.copy_(wo)
    step(blocks, make_rows(2 * B, Hq, d, 91), make_rows(2 * B, Hkv, d, 92), make_rows(2 * B, Hkv, d, 93))
    m.bdlm_sync_status(ws)


@pytest.mark.parametrize("B", [1, 40])
def test_captured_step_follows_lengths_and_pages(lib, B):
    """A graph of attend + weigh + append + length update, replayed: equal,
    bit for bit, to the same calls made one by one."""
    m = lib
    Hq, Hkv, d, page = 8, 2, 64, 16
    c, _ = make_cache([70, 9], 70 + 6 * B, Hkv, d, page, seed=71)
    make = lambda: (device_cache(m, torch, c), torch.zeros((2, Hkv, c["table"].shape[1] * page), device="cuda"))
    rows = lambda s: [to_dev(make_rows(2 * B, H, d, s + i), torch) for i, H in enumerate((Hq, Hkv, Hkv))]
    side = torch.cuda.Stream()

    def one(cache, W, ws, x, out):
        m.bdlm_attn_cached(*x, cache, out=out, workspace=ws)
        m.bdlm_cache_weights(x[0], out[1], cache, W, workspace=ws)
        nl = m.bdlm_cache_append(cache, x[1], x[2], workspace=ws)
        cache.lens.copy_(nl)

    outs = lambda: (torch.empty((2 * B, Hq, d), dtype=torch.bfloat16, device="cuda"),
                    torch.empty((Hq, 2 * B), device="cuda"))
    ca, Wa = make()
    cb, Wb = make()
    wa, wb, oa, ob, x = (*(m.bdlm_cache_workspace(k, Hq, B) for k in (ca, cb)), outs(), outs(), rows(0))
    lens0 = cb.lens.clone()
    saved = [t.clone() for t in (cb.k8.view(torch.uint8), cb.v8.view(torch.uint8), cb.k_scale, cb.v_scale)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        one(cb, Wb, wb, x, ob)
    for t, s in zip((cb.k8.view(torch.uint8), cb.v8.view(torch.uint8), cb.k_scale, cb.v_scale), saved):
        t.copy_(s)
    cb.lens.copy_(lens0)
    Wb.zero_()
    for k in range(4):
        for t, s in zip(x, rows(10 * k)):
            t.copy_(s)
        one(ca, Wa, wa, x, oa)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa[0], ob[0]) and torch.equal(oa[1], ob[1]) and torch.equal(Wa, Wb)
        assert torch.equal(ca.lens, cb.lens) and torch.equal(ca.k8.view(torch.uint8), cb.k8.view(torch.uint8))
    m.bdlm_sync_status(wa)
    m.bdlm_sync_status(wb)


def test_calls_on_a_given_stream(lib):
    m = lib
    c, _ = make_cache([400, 30], 400, 2, 64, 16, seed=81)
    cache = device_cache(m, torch, c)
    Q = to_dev(make_rows(2, 8, 64, 1), torch)
    ref = m.bdlm_attn_cached(Q, None, None, cache)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = m.bdlm_attn_cached(Q, None, None, cache, stream=side)  # its workspace and outputs are made by the call
    side.synchronize()
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])


def test_shared_prefix_pages(lib):
    """Two sequences whose tables name the same pages read the same keys."""
    m = lib
    c, _ = make_cache([64, 64], 64, 2, 64, 16, seed=83)
    c["table"][1] = c["table"][0]
    Q = make_rows(2, 8, 64, 1)
    O, LSE = m.bdlm_attn_cached(to_dev(Q, torch), None, None, device_cache(m, torch, c), o_dtype=torch.float32)
    check_attn(O, LSE, co.attn(c, Q, None, None, offsets_of([1, 1]), 0.125), 64, False)


def test_binding_refuses(lib):
    m = lib
    c, (dst,) = make_cache([10], 16, 2, 64, 16, seed=85, sets=2)
    cache = device_cache(m, torch, c)
    Q = to_dev(make_rows(1, 4, 64, 1), torch)
    with pytest.raises(ValueError):
        m.bdlm_attn_cached(Q.float(), None, None, cache)
    with pytest.raises(ValueError):
        m.bdlm_attn_cached(torch.cat([Q, Q], 2)[:, :, ::2], None, None, cache)  # not contiguous
    with pytest.raises(ValueError):
        m.bdlm_attn_cached(Q, Q[:, :2].contiguous(), None, cache)
    with pytest.raises(ValueError):
        m.bdlm_attn_cached(Q, None, None, cache, torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        m.bdlm_attn_cached(Q, None, None, cache, o_dtype=torch.float16)
    with pytest.raises(m.BdlmError):
        m.bdlm_cache_append(cache, Q[:, :2].contiguous(), Q[:, :2].contiguous(), lens_out=cache.lens)
    with pytest.raises(AttributeError):
        cache.lens = cache.lens
    W = torch.zeros((1, 2, 16), device="cuda")
    with pytest.raises(m.BdlmError):
        m.bdlm_cache_evict(cache, W, cache.page_table, 4)
    with pytest.raises(m.BdlmError):
        m.bdlm_cache_evict(cache, W, torch.from_numpy(dst).cuda(), 4, weights_out=W)
