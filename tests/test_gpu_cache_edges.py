"""The 8-bit cache's calls where their number formats end (GPU): a dominant
key, blocks of zeros, tiny queries, channels of unlike size, sequences without
new rows; and what the status words say.  Tolerances as in test_gpu_cache.py,
with the floors that the header gives added where a test reaches them."""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle.cache_oracle as co
from structured_mask_attention_gb300.inputs import bf16_round
from tests.cache_util import device_cache, host_codes, make_cache, make_rows, offsets_of
from tests.parity_util import to_dev
from tests.test_gpu_cache import HALF, check_attn, lib, score_error  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def sink_case(L, d, rows, nats, seed, at=0, value=0.0):
    """One key of ``nats`` more than the others' mean score for every query, its value ``value`` times
    the others'; 2 heads on one KV head, pages of 64."""
    c, _ = make_cache([L], L, 1, d, 64, seed)
    Q = make_rows(rows, 2, d, seed + 1)
    pages = c["table"][0, : -(-L // 64)]
    c["k8"][pages, :, :, :8] = 0                     # channels 0 to 7 are the sink's alone
    pg, slot = c["table"][0, at // 64], at % 64
    Q[:, :, :8] = bf16_round(np.float32(nats * math.sqrt(d) / (8 * 1.25)))
    c["k8"][pg, 0, slot] = 0
    c["k8"][pg, 0, slot, :8] = co.encode(1.25 / c["ks"][pg, 0])
    c["v8"][pg, 0, slot] = co.encode(co.E4M3[c["v8"][pg, 0, slot]] * value)
    return c, Q


@pytest.mark.parametrize("rows", [1, 16, 40, 150])   # mma.sync in tiles of 16 and 32, tcgen05 split and in pairs
@pytest.mark.parametrize("nats,at", [(14, 0), (18, 0), (20, 0), (18, 3900)])
@pytest.mark.parametrize("d", [64, 128])
def test_attn_sink_without_a_value(lib, rows, nats, at, d):
    """The others' weights, 2^-20 to 2^-29 of the largest one, are all of O.  (The
    row's 4096 keys are in one CTA's piece.)"""
    m = lib
    n = 152 * (2 if 2 * rows <= 32 else 1)           # sequences on the same pages: one or two for each CTA
    c, Q = sink_case(4096, d, rows, nats, seed=nats + rows, at=at)
    c["table"], c["lens"] = np.repeat(c["table"], n, 0), np.repeat(c["lens"], n)
    O, LSE = m.bdlm_attn_cached(to_dev(np.concatenate([Q] * n), torch), None, None, device_cache(m, torch, c))
    one = {**c, "table": c["table"][:1], "lens": c["lens"][:1]}
    ref = co.attn(one, Q, None, None, offsets_of([rows]), 1 / math.sqrt(d))
    # of O: bf16's rounding, 2^-9 at most in the mean, and each weight's in fp16, evenly spread and unlike in sign, 2^-11
    # of it and at least 2^-25 of the row's largest weight 1 times 2^9 (pages' scales: at most 4 times that): its root
    # mean square, by that of the weights
    z = Q[0, 0].astype(np.float64) @ co.tokens(one, "k", 0, 0).T / math.sqrt(d)
    p = np.delete(np.exp(z - z.max()), at)
    limit = math.sqrt(2.0 ** -18 + 2.0 ** -22 + (4 * 2.0 ** -34 / math.sqrt(3) / math.sqrt((p ** 2).mean())) ** 2)
    for s in (0, n // 2, n - 1):
        o = O[s * rows:(s + 1) * rows]
        check_attn(o, LSE[:, s * rows:(s + 1) * rows], ref, d, True)
        rel = np.linalg.norm(o.double().cpu().numpy() - ref[0]) / np.linalg.norm(ref[0])
        print(f"  O off by {rel:.2e} of its size")
        assert rel <= 1.25 * limit


@pytest.mark.parametrize("rows", [1, 16, 40, 150])
@pytest.mark.parametrize("value", [0.0, 0.02, 1.0])
def test_attn_fp32_of_weights_far_apart(lib, rows, value):
    """fp32 outputs: a weight enters to 2^-22 of itself and 2^-34 of the row's
    largest weight times its value block's scale."""
    m = lib
    d, L = 128, 4096
    n = 152 * (2 if 2 * rows <= 32 else 1)
    c, Q = sink_case(L, d, rows, 16, seed=7 + rows, value=value)
    c["table"], c["lens"] = np.repeat(c["table"], n, 0), np.repeat(c["lens"], n)
    O, LSE = m.bdlm_attn_cached(to_dev(np.concatenate([Q] * n), torch), None, None, device_cache(m, torch, c),
                                o_dtype=torch.float32)
    one = {**c, "table": c["table"][:1], "lens": c["lens"][:1]}
    Or, Lr, A, E = co.attn(one, Q, None, None, offsets_of([rows]), 1 / math.sqrt(d))
    # the floor: 2^-34 (largest p vs) |code_j| summed over j; scales differ by 4 at most, p <= 1
    floor = 4 * 2.0 ** -34 * np.abs(co.tokens(one, "v", 0, 0)).sum(0)
    ds = score_error(d, E)
    for s in (0, n - 1):
        o = O[s * rows:(s + 1) * rows].double().cpu().numpy()
        tol = (2.0 ** -22 + 2 * ds.T[:, :, None]) * A + floor
        worst = (np.abs(o - Or) / tol).max()
        rel = np.linalg.norm(o - Or) / np.linalg.norm(Or)
        print(f"  O {worst:.3f} of its tolerance, off by {rel:.2e} of its size")
        assert worst <= 1
        lse = LSE[:, s * rows:(s + 1) * rows].double().cpu().numpy()
        assert (np.abs(lse - Lr) <= ds + 2.0 ** -22 * (1 + np.abs(Lr))).all()


@pytest.mark.parametrize("rows", [1, 20, 40, 150])
@pytest.mark.parametrize("page,L", [(128, 168), (32, 128 + 32 + 7)])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
def test_attn_tiny_queries_on_a_block_of_zeros(lib, rows, page, L, o_dtype):
    """A key block of zeros has the scale 2^-64; with a query of 2^-90 the product
    of both scales is below the smallest fp32 number, in a tile that ends inside."""
    m = lib
    c, _ = make_cache([L], L, 1, 64, page, seed=3)
    last = c["table"][0, 128 // page:]
    c["k8"][last], c["ks"][last] = 0, 2.0 ** -64
    Q = bf16_round(make_rows(rows, 2, 64, 1) * np.float32(2.0 ** -90))
    O, LSE = m.bdlm_attn_cached(to_dev(Q, torch), None, None, device_cache(m, torch, c), o_dtype=o_dtype)
    check_attn(O, LSE, co.attn(c, Q, None, None, offsets_of([rows]), 0.125), 64, o_dtype == torch.bfloat16)


@pytest.mark.parametrize("rows", [1, 20, 40, 150])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("factor", [30.0, 100.0, 1000.0])
def test_attn_and_weights_of_a_channel_of_another_size(lib, rows, d, factor):
    """One channel of the queries is ``factor`` times the others."""
    m = lib
    L = 700
    c, _ = make_cache([L], L, 1, d, 32, seed=5)
    Q = make_rows(rows, 2, d, 1)
    Q[:, :, 5] = bf16_round(Q[:, :, 5] * np.float32(factor))
    sc, cache = 1 / math.sqrt(d), device_cache(m, torch, c)
    sc *= 0.25 if factor < 200 else 0.025
    O, LSE = m.bdlm_attn_cached(to_dev(Q, torch), None, None, cache, scale=sc, o_dtype=torch.float32)
    ref = co.attn(c, Q, None, None, offsets_of([rows]), sc)
    check_attn(O, LSE, ref, d, False)
    W = torch.zeros((1, 1, c["table"].shape[1] * 32), device="cuda")
    m.bdlm_cache_weights(to_dev(Q, torch), torch.from_numpy(ref[1].astype(np.float32)).cuda(), cache, W, scale=sc)
    Wr, E = co.weights(c, Q, ref[1].astype(np.float32), offsets_of([rows]), sc, np.zeros(W.shape, np.float32))
    rel = score_error(d, E) + 2.0 ** -23 * (1 + np.abs(ref[1]).max()) + (2 * rows + 4) * 2.0 ** -24
    worst = (np.abs(W.double().cpu().numpy() - Wr) / (rel * Wr + 2.0 ** -24)).max()
    print(f"  weights {worst:.3f} of their tolerance")
    assert worst <= 1


@pytest.mark.parametrize("rows,Hq,local,chain", [(32, 1, True, 3), (16, 2, True, 3), (32, 1, False, 2)])
@pytest.mark.parametrize("L", [0, 3000])
def test_attn_fp32_output_with_own_keys(lib, rows, Hq, local, chain, L):
    """mma.sync tiles, fp32 O: the tensor cores cut a sum off by up to 2^-23 of
    it, always towards zero, 2/3 of its last size in the mean; the products of 16
    keys, two (own keys: three) of their weights' parts, are added to O by the
    threads, rounded.  2^-21 for the weights' and scores' own errors."""
    m = lib
    d, n = 128, 40
    c, _ = make_cache([L], max(L, 1), 1, d, 64, seed=93)
    c["table"], c["lens"] = np.repeat(c["table"], n, 0), np.repeat(c["lens"], n)
    if not local and not L:
        return
    Q, K, V = (make_rows(n * rows, H, d, 3 + i) for i, H in enumerate((Hq, 1, 1)))
    kv = (K, V) if local else (None, None)
    dkv = [None if x is None else to_dev(x, torch) for x in kv]
    O, LSE = m.bdlm_attn_cached(to_dev(Q, torch), *dkv, device_cache(m, torch, c), o_dtype=torch.float32)
    ref = co.attn(c, Q, *kv, offsets_of([rows] * n), 1 / math.sqrt(d))
    check_attn(O, LSE, ref, d, False)
    diff = O.double().cpu().numpy() - ref[0]
    rel = math.sqrt((diff ** 2).sum() / (ref[0] ** 2).sum())
    print(f"  O off by {rel:.2e} of its size")
    assert rel <= chain * 2.0 ** -23 * 2 / 3 + 2.0 ** -21


@pytest.mark.parametrize("rows", [1, 16, 40, 150])
@pytest.mark.parametrize("size", [2.0 ** 16, 2.0 ** 22, 2.0 ** 26])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
def test_attn_scores_beyond_fp32s_fractions(lib, rows, size, o_dtype):
    """Scores of 2^20 and more, whose roundings are of a binary order or more: a row
    is a mean of values still (which keys share it is below fp32's resolution)."""
    m = lib
    c, _ = make_cache([700], 700, 1, 64, 16, seed=23)
    Q, K, V = (make_rows(rows, H, 64, 1 + i) for i, H in enumerate((2, 1, 1)))
    Q = bf16_round(Q * np.float32(size))
    cache, dev = device_cache(m, torch, c), lambda x: to_dev(x, torch)
    for kv in ((None, None), (dev(K), dev(V))):
        O, LSE = m.bdlm_attn_cached(dev(Q), *kv, cache, o_dtype=o_dtype)
        assert torch.isfinite(O).all() and torch.isfinite(LSE).all()
        ref = co.attn(c, Q, *((K, V) if kv[0] is not None else (None, None)), offsets_of([rows]), 0.125)
        # the row's largest score, in natural units
        assert (np.abs(LSE.double().cpu().numpy() - ref[1]) <= score_error(64, ref[3]) + 2.0 ** -22 * np.abs(ref[1])).all()
        v = np.concatenate([co.tokens(c, "v", 0, 0)] + ([V[:, 0]] if kv[0] is not None else []))
        assert (O.double().cpu().numpy() <= v.max(0) * (1 + HALF) + 1e-3).all()
        assert (O.double().cpu().numpy() >= v.min(0) * (1 + HALF) - 1e-3).all()


@pytest.mark.parametrize("rows", [4, 300])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_weights_leave_rows_of_lse_minus_infinity_out(lib, rows, d, value):
    """A padded batch: rows marked by LSE = -inf, whose queries hold anything."""
    m = lib
    c, _ = make_cache([300], 300, 2, d, 64, seed=27)
    Q = make_rows(rows, 4, d, 1)
    off = offsets_of([rows])
    LSE = co.attn(c, Q, None, None, off, 0.1)[1].astype(np.float32)
    pad = np.arange(rows) % 3 == 1
    LSE[:, pad] = -np.inf
    Wr, E = co.weights(c, Q, LSE, off, 0.1, np.zeros((1, 2, 320), np.float32))
    Q[pad] = value
    W = torch.zeros((1, 2, 320), device="cuda")
    m.bdlm_cache_weights(to_dev(Q, torch), torch.from_numpy(LSE).cuda(), device_cache(m, torch, c), W, scale=0.1)
    rel = score_error(d, E) + 2.0 ** -23 * (1 + np.abs(LSE[:, ~pad]).max()) + (2 * rows + 4) * 2.0 ** -24
    assert (np.abs(W.double().cpu().numpy() - Wr) <= rel * Wr + 2.0 ** -24).all()


@pytest.mark.parametrize("rows", [5, 20, 33, 60, 150, 300])  # (60 and more: own tiles of their own; 150, 300: several)
@pytest.mark.parametrize("factor", [1.0, 2.0 ** -40, 2.0 ** 40])
@pytest.mark.parametrize("L", [0, 200])
def test_attn_own_keys_count_as_near_as_cached_ones(lib, rows, factor, L):
    """bf16 outputs: an own key's weight is off by 2^-11 at most, its values, of
    any size and unlike within a tile, by 2^-34 of the tile's largest."""
    m = lib
    d, Hq, n = 64, 2, 3
    c, _ = make_cache([L] * n, max(L, 1), 1, d, 64, seed=17)
    T = n * rows
    Q, K = (make_rows(T, H, d, i) for i, H in ((1, Hq), (2, 1)))
    V = make_rows(T, 1, d, 3) * np.exp2(np.random.default_rng(4).integers(-20, 1, (T, 1, d))).astype(np.float32)
    V = bf16_round(V * np.float32(factor))
    if L:
        c["vs"] *= np.float32(factor)
    O, LSE = m.bdlm_attn_cached(*(to_dev(x, torch) for x in (Q, K, V)), device_cache(m, torch, c))
    Or, Lr, A, E = co.attn(c, Q, K, V, offsets_of([rows] * n), 1 / math.sqrt(d))
    ds = score_error(d, E)
    assert (np.abs(LSE.double().cpu().numpy() - Lr) <= ds + 2.0 ** -22 * (1 + np.abs(Lr))).all()
    big = max(np.abs(V).max(), 448 * float(np.nanmax(c["vs"])) if L else 0.0)
    tol = (2.0 ** -11 + 2 * ds.T[:, :, None]) * A + HALF * np.abs(Or) + 2.0 ** -33 * big * (L + rows)
    worst = (np.abs(O.double().cpu().numpy() - Or) / tol).max()
    print(f"  O {worst:.3f} of its tolerance")
    assert worst <= 1


@pytest.mark.parametrize("rows", [10, 20, 40, 150])
def test_attn_own_values_that_are_not_finite_or_zero(lib, rows):
    """An infinite value reaches its column of its own sequence's rows; zeros are zeros."""
    m = lib
    d = 64
    c, _ = make_cache([70, 70, 0], 128, 1, d, 64, seed=19)
    Q, K, V = (make_rows(3 * rows, H, d, 1 + i) for i, H in enumerate((2, 1, 1)))
    V[3, 0, 7], V[5, 0, 9] = math.inf, math.nan
    V[2 * rows:] = 0.0
    cache = device_cache(m, torch, c)
    for o_dtype in (torch.bfloat16, torch.float32):
        O, LSE = m.bdlm_attn_cached(*(to_dev(x, torch) for x in (Q, K, V)), cache, o_dtype=o_dtype)
        assert torch.isfinite(LSE).all()
        if o_dtype == torch.bfloat16:
            assert (O[:rows, :, 7] == math.inf).all()
        else:  # (on tcgen05 the second part of a weight meets it too, and may be 0)
            assert not torch.isfinite(O[:rows, :, 7]).any()
        assert torch.isnan(O[:rows, :, 9]).all()
        fine = np.setdiff1d(np.arange(d), [7, 9])
        W = V.copy()
        W[3, 0, 7] = W[5, 0, 9] = 0.0
        ref = co.attn(c, Q, K, W, offsets_of([rows] * 3), 0.125)
        check_attn(O[rows:], LSE[:, rows:], (ref[0][rows:], ref[1][:, rows:], ref[2][rows:], ref[3][:, rows:]), d,
                   o_dtype == torch.bfloat16)
        check_attn(O[:rows][:, :, fine], LSE[:, :rows], (ref[0][:rows][:, :, fine], ref[1][:, :rows],
                                                         ref[2][:rows][:, :, fine], ref[3][:, :rows]), d,
                   o_dtype == torch.bfloat16)
        assert (O[2 * rows:] == 0).all()


@pytest.mark.parametrize("scale", [2.0 ** -70, math.nan])
@pytest.mark.parametrize("page,d", [(16, 64), (64, 128), (128, 128)])
def test_append_leaves_a_sequence_without_rows_alone(lib, scale, page, d):
    """No new rows: the partly filled last page (it may be another sequence's
    too) keeps its codes and scale, whatever that is."""
    m = lib
    c, _ = make_cache([5, 3, 9], 2 * page, 2, d, page, seed=4)
    for s in (0, 2):
        c["ks"][c["table"][s, 0]] = c["vs"][c["table"][s, 0]] = scale
    K = make_rows(7, 2, d, 1)
    off = np.array([0, 0, 7, 7], np.int32)
    cache = device_cache(m, torch, c)
    ws = m.bdlm_cache_workspace(cache)
    cache.page_table[2, 0] = 10 ** 6                 # nor is its table looked at
    got = m.bdlm_cache_append(cache, to_dev(K, torch), to_dev(K, torch), torch.from_numpy(off).cuda(), workspace=ws)
    m.bdlm_sync_status(ws)
    assert got.tolist() == [5, 10, 9]
    co.append(c, K, K, off)
    for w in ("k", "v"):
        assert np.array_equal(host_codes(getattr(cache, w + "8")), c[w + "8"])
        assert np.array_equal(getattr(cache, w + "_scale").cpu().numpy(), c[w + "s"], equal_nan=True)


def test_a_timeout_is_reported_whatever_the_contents_were(lib):
    """Contents out of range and an expired wait have a word each: neither hides
    the other, and a timeout (here: its code, written as a kernel would) is what
    the report names."""
    m = lib
    c, _ = make_cache([60], 64, 1, 64, 16, seed=51)
    cache = device_cache(m, torch, c)
    ws = m.bdlm_cache_workspace(cache, 2, 1)
    words = ws[:64].view(torch.int32)
    cache.page_table[0, 1] = -5
    Q = to_dev(make_rows(1, 2, 64, 1), torch)
    def call():
        m.bdlm_attn_cached(Q, None, None, cache, workspace=ws)
        torch.cuda.synchronize()
    call()
    assert int(words[0]) == 0                        # free for the first expired wait
    with pytest.raises(m.BdlmError, match="page id"):
        m.bdlm_sync_status(ws)
    for first in (True, False):
        if not first:
            call()
        words[0] = 0x7100 | 33
        if first:
            call()
        with pytest.raises(m.BdlmError, match="wait site 33") as e:
            m.bdlm_sync_status(ws)
        assert e.value.status == 7 and "page id" in str(e.value)
        m.bdlm_sync_status(ws)                       # both are read once


def test_captured_eviction(lib):
    """A graph of weigh + evict, replayed on other weights and lengths."""
    m = lib
    keep = 40
    c, (dst,) = make_cache([300, 90], 320, 2, 64, 16, seed=71, sets=2)
    cache, ddst = device_cache(m, torch, c), torch.from_numpy(dst).cuda()
    ws = m.bdlm_cache_workspace(cache, 4, 1, keep)
    W = torch.zeros((2, 2, c["table"].shape[1] * 16), device="cuda")
    out = (torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros_like(W),
           torch.zeros((2, 2, keep), dtype=torch.int32, device="cuda"))
    call = lambda: m.bdlm_cache_evict(cache, W, ddst, keep, 2, 8, *out, workspace=ws)
    codes = lambda: [t.clone() for t in (cache.k8.view(torch.uint8), cache.v8.view(torch.uint8), cache.k_scale,
                                         cache.v_scale)]
    saved = codes()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call()
    for k in range(4):
        rng = np.random.default_rng(k)
        Wn = rng.random(W.shape, dtype=np.float32)
        lens = np.array([300 - 61 * k, 90 - 20 * k], np.int32)
        W.copy_(torch.from_numpy(Wn))
        cache.lens.copy_(torch.from_numpy(lens))
        for t, s in zip((cache.k8.view(torch.uint8), cache.v8.view(torch.uint8), cache.k_scale, cache.v_scale), saved):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        h = {x: v.copy() for x, v in c.items()}
        h["lens"] = lens
        rl, rw, rk = co.evict(h, Wn, dst, keep, 2, 8)
        assert out[0].tolist() == rl.tolist() and np.array_equal(out[1].cpu().numpy(), rw)
        assert np.array_equal(out[2].cpu().numpy(), rk)
        for w in ("k", "v"):
            assert np.array_equal(host_codes(getattr(cache, w + "8")), h[w + "8"])
    m.bdlm_sync_status(ws)
