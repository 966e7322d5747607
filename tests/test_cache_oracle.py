"""The 8-bit cache's oracle, pinned without its own formulas (CPU)."""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle.bdlm_oracle as orc
import oracle.cache_oracle as co
from tests.cache_util import make_cache, make_rows, offsets_of

torch = pytest.importorskip("torch")


def test_codes_are_torch_e4m3():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(v, co.E4M3, equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 4000), rng.standard_normal(4000), rng.standard_normal(4000) * 2.0 ** -8,
                        co._POS, (co._POS[1:] + co._POS[:-1]) / 2, [0.0, -0.0, 447.9, 448.0]]).astype(np.float32)
    assert np.array_equal(torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), co.encode(x))
    assert co.encode([1e9, -1e9, np.nan]).tolist()[:2] == [126, 254]


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (449.0, 2.0), (1.75, 2.0 ** -8), (1.7578125, 2.0 ** -7),
                                        (0.0, 2.0 ** -64), (1e-30, 2.0 ** -64), (3e38, 2.0 ** 120)])
def test_block_scale(amax, scale):
    assert co.block_scale(np.array([0.0, -amax])) == scale


def test_block_scale_of_values_that_are_not_finite():
    assert math.isnan(co.block_scale(np.array([1.0, np.inf]))) and math.isnan(co.block_scale(np.array([np.nan])))


def test_attention_is_the_corrupted_stream_of_the_two_stream_oracle():
    """A block against its clean prefix from a cache = the corrupted rows of the
    training mask, on the values that the codes stand for."""
    L, B, Hq, Hkv, d = 96, 32, 4, 2, 64
    X = {k: make_rows(L, H, d, i) for i, (k, H) in enumerate((("Qc", Hq), ("Kc", Hkv), ("Vc", Hkv), ("Qn", Hq),
                                                             ("Kn", Hkv), ("Vn", Hkv)))}
    for b in range(L // B):
        c, _ = make_cache([0], L, Hkv, d, 16, seed=b)
        c["lens"] = co.append(c, X["Kc"][: b * B], X["Vc"][: b * B], offsets_of([b * B]))
        kc, vc = X["Kc"].astype(np.float64).copy(), X["Vc"].astype(np.float64).copy()
        for h in range(Hkv):
            kc[: b * B, h], vc[: b * B, h] = co.tokens(c, "k", 0, h), co.tokens(c, "v", 0, h)
        sl = slice(b * B, (b + 1) * B)
        O, LSE, _, _ = co.attn(c, X["Qn"][sl], X["Kn"][sl], X["Vn"][sl], offsets_of([B]), 0.125)
        x64 = {k: v.astype(np.float64) for k, v in X.items()}
        ref = orc.fwd_brute(x64["Qc"], kc, vc, x64["Qn"], x64["Kn"], x64["Vn"], B, 0.125)
        assert np.abs(O - ref[1][sl]).max() < 1e-12 and np.abs(LSE - ref[3][:, sl]).max() < 1e-12


def test_append_rounds_each_value_to_its_blocks_step():
    rng = np.random.default_rng(1)
    c, _ = make_cache([5, 0], 64, 2, 64, 16, seed=2)
    before = [co.tokens(c, "k", 0, h) for h in range(2)]
    K = make_rows(30, 2, 64, 3) * np.exp(rng.standard_normal((30, 1, 1)).astype(np.float32))
    c["lens"] = co.append(c, K, K, offsets_of([20, 10]))
    assert c["lens"].tolist() == [25, 10]
    for s, a, b, L in ((0, 0, 20, 5), (1, 20, 30, 0)):
        for h in range(2):
            got, want = co.tokens(c, "k", s, h)[L:], K[a:b, h]
            step = np.repeat([c["ks"][c["table"][s, i // 16], h] for i in range(L, L + b - a)], 64).reshape(got.shape)
            # half a step: 2^-4 relative, and half of the smallest step below 2^-6 scale
            assert (np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * step)).all()
    for h in range(2):  # old tokens: unchanged, or rounded once more to a coarser scale
        assert (np.abs(co.tokens(c, "k", 0, h, 5) - before[h]) <= 2.0 ** -4 * np.abs(before[h]) + 2.0 ** -10 *
                c["ks"][c["table"][0, 0], h]).all()


def test_weights_add_up_to_the_rows():
    """Without an own block every row gives a total weight of one per head."""
    c, _ = make_cache([37, 20], 48, 2, 64, 16, seed=4)
    Q, off = make_rows(5, 4, 64, 5), offsets_of([2, 3])
    LSE = co.attn(c, Q, None, None, off, 0.125)[1]
    W, _ = co.weights(c, Q, LSE, off, 0.125, np.zeros((2, 2, 48)))
    assert np.allclose(W.sum(2), [[2 * 2, 2 * 2], [3 * 2, 3 * 2]], atol=1e-12)
    assert (W[0, :, 37:] == 0).all()


def test_evict_keeps_sinks_recent_and_the_heaviest():
    c, (dst,) = make_cache([10], 16, 1, 64, 16, seed=6, sets=2)
    W = np.zeros((1, 1, 16), np.float32)
    W[0, 0, :10] = [0, 5, 1, 7, 1, 1, 9, 0, 0, 0]
    x = co.tokens(c, "k", 0, 0)
    lens, Wout, kept = co.evict(c, W, dst, 6, 1, 1)
    assert kept[0, 0].tolist() == [0, 1, 2, 3, 6, 9] and lens.tolist() == [6]
    assert Wout[0, 0, :7].tolist() == [0, 5, 1, 7, 9, 0, 0]
    c["table"], c["lens"] = dst, lens
    assert np.abs(co.tokens(c, "k", 0, 0) - x[[0, 1, 2, 3, 6, 9]]).max() <= 2.0 ** -10 * c["ks"][dst[0, 0], 0]


def test_a_query_is_the_sum_of_its_two_8_bit_parts():
    """What the tensor-core kernels multiply for a query row: its values, scaled
    by a power of two into [128, 256), as the nearest e4m3 values plus the e5m2
    values of what those left.  Exact down to 2^-13 of the largest, off by 2^-21 below."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn((20000, 64), generator=g) * torch.exp2(torch.rand((20000, 64), generator=g) * -30)
    x[:, 0] = torch.randn(20000, generator=g) * 4
    x = x.bfloat16().float()
    top = x.abs().amax(1, keepdim=True)
    v = (x * torch.exp2(7 - torch.floor(torch.log2(top)))).half().float()
    hi = v.to(torch.float8_e4m3fn).float()
    lo = (v - hi).half().to(torch.float8_e5m2).float()
    off = (v.double() - hi.double() - lo.double()).abs()
    largest = v.abs().amax(1, keepdim=True).double()
    assert (largest >= 128).all() and (largest < 256).all()
    assert (off[v.abs() >= 2.0 ** -13 * largest] == 0).all() and (off <= 2.0 ** -21 * largest).all()
    # every significand of 8 bits, signs and all exponents from e4m3's smallest normal one on
    v = (torch.arange(128, 256).float()[None] * torch.exp2(torch.arange(-13, 1).float())[:, None]).reshape(-1)
    v = torch.cat([v, -v])
    hi = v.to(torch.float8_e4m3fn).float()
    assert torch.equal(hi + (v - hi).to(torch.float8_e5m2).float(), v)
