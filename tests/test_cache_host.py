"""Host checks of the 8-bit cache's calls: argument validation before anything
reaches a device (CPU)."""
from __future__ import annotations

import ctypes

import pytest

import structured_mask_attention_gb300 as m
from structured_mask_attention_gb300.build import build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    build()
    return m.load_library()


def _cache(**kw):
    f = dict(k8=0x100000, v8=0x200000, k_scale=0x300000, v_scale=0x310000, page_table=0x320000, lens=0x330000,
             n_pages=64, n_seqs=4, max_pages=8, page=16, Hkv=2, d=64)
    f.update(kw)
    return m._CacheStruct(*f.values())


def _attn(lib, cache=None, Q=0x400000, K=0x500000, V=0x600000, off=None, rows=4, max_rows=1, Hq=4, scale=0.125,
          O=0x700000, dt=0, LSE=0x800000, ws=0x900000, nb=1 << 30):
    c = _cache() if cache is None else cache
    return lib.bdlm_attn_cached(Q, K, V, ctypes.cast(ctypes.pointer(c), ctypes.c_void_p), off, rows, max_rows, Hq,
                                scale, O, dt, LSE, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=96), 2), (dict(page=8), 2), (dict(page=48), 2), (dict(page=256), 2), (dict(Hkv=0), 2),
    (dict(n_seqs=0), 2), (dict(n_seqs=65536), 2), (dict(n_pages=0), 2), (dict(n_pages=1 << 31), 2),
    (dict(n_pages=(1 << 30) + 1), 2),                  # n_pages * Hkv passes 2^31
    (dict(max_pages=0), 2), (dict(max_pages=(1 << 26) + 1), 2),
    (dict(k8=None), 1), (dict(v_scale=None), 1), (dict(lens=None), 1), (dict(v8=0x200008), 3),
    (dict(page_table=0x320002), 3),
])
def test_cache_is_checked(lib, kw, status):
    assert _attn(lib, cache=_cache(**kw)) == status, m.bdlm_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=3), 2), (dict(Hq=0), 2), (dict(scale=0.0), 1), (dict(scale=float("inf")), 1), (dict(dt=2), 1),
    (dict(K=None), 1), (dict(V=None), 1), (dict(Q=None), 1), (dict(Q=0x400008), 3), (dict(O=0x700004), 3),
    (dict(LSE=None), 1), (dict(ws=None), 4), (dict(nb=256), 4), (dict(ws=0x900008), 3),
    (dict(rows=5), 2),                                 # not n_seqs * max_rows, and no row_offsets
    (dict(max_rows=0), 2), (dict(rows=-1), 2), (dict(max_rows=(1 << 24) + 1), 2), (dict(off=0x320001), 3),
])
def test_attn_is_checked(lib, kw, status):
    assert _attn(lib, **kw) == status, m.bdlm_last_error()


@pytest.mark.parametrize("kw", [dict(O=0x400000), dict(O=0x400000 - 2048 + 16), dict(O=0x500000), dict(O=0x600000 + 512),
                                dict(LSE=0x700000), dict(O=0x400000 - 4096 + 16, dt=1)])
def test_attn_outputs_lie_apart(lib, kw):
    """4 rows of 4 heads (K, V: 2) of 64: 2048 (1024) bytes, an fp32 O 4096."""
    assert _attn(lib, **kw) == 1 and "overlaps" in m.bdlm_last_error(), m.bdlm_last_error()


def test_weights_units_fit_32_bits(lib):
    c = _cache(max_pages=1 << 26, page=16, Hkv=1)     # 2^23 key tiles
    call = lambda Hq: lib.bdlm_cache_weights(0x400000, 0x500000, ctypes.cast(ctypes.pointer(c), ctypes.c_void_p),
                                             0x340000, 4, 1 << 14, Hq, 0.125, 0x700000, 0x900000, 256, None)
    assert call(2) == 2 and "2^30" in m.bdlm_last_error()  # by 2^8 row tiles: 2^31
    if not torch.cuda.is_available():
        assert call(1) in (5, 6)                           # 2^30 pass (and there is no device)


@pytest.mark.parametrize("kw", [dict(LSE=0x400000), dict(LSE=0x500000 - 60), dict(LSE=0x600000 + 1020)])
def test_attn_lse_lies_apart_from_inputs(lib, kw):
    """4 rows of 4 heads: 64 bytes of LSE; Q, K, V of 2048, 1024 and 1024."""
    assert _attn(lib, **kw) == 1 and "LSE overlaps" in m.bdlm_last_error(), m.bdlm_last_error()


@pytest.mark.parametrize("call,kw", [
    ("append", dict(off=0x340000, lens_out=0x340010)), ("append", dict(lens_out=0x320000 + 4 * 31)),
    ("weights", dict(W=0x400000 + 2032)), ("weights", dict(W=0x500000 - 4080)),
    ("evict", dict(lens=0x350000 + 4 * 31)), ("evict", dict(kept=0x700000 + 4092)), ("evict", dict(kept=0x800000 - 2044)),
    ("evict", dict(dst=0x320000 + 4 * 31)),
])
def test_outputs_lie_apart_from_inputs(lib, call, kw):
    """4 sequences, 2 KV heads, 8 pages of 16: tables of 128 bytes, weights of 4096, kept (64) of 2048."""
    c = _cache()
    ref = ctypes.cast(ctypes.pointer(c), ctypes.c_void_p)
    a = dict(off=None, lens_out=0x348000, Q=0x400000, LSE=0x500000, W=0x700000, dst=0x350000, lens=0x340000, kept=None)
    a.update(kw)
    if call == "append":
        s = lib.bdlm_cache_append(0x400000, 0x500000, ref, a["off"], 4, 1, a["lens_out"], 0x900000, 256, None)
    elif call == "weights":
        s = lib.bdlm_cache_weights(a["Q"], a["LSE"], ref, None, 4, 1, 4, 0.125, a["W"], 0x900000, 256, None)
    else:
        s = lib.bdlm_cache_evict(ref, a["W"], a["dst"], 64, 4, 8, a["lens"], 0x800000, a["kept"], 0x900000, 1 << 20, None)
    assert s == 1 and "overlaps" in m.bdlm_last_error(), (s, m.bdlm_last_error())


def test_no_rows_is_no_work(lib):
    assert _attn(lib, off=0x340000, rows=0, Q=None, K=None, V=None) == 0


def test_null_cache(lib):
    assert lib.bdlm_cache_append(1 << 20, 1 << 20, None, None, 4, 1, None, 1 << 20, 256, None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(lens_out=0x330000), 1), (dict(lens_out=0x330008), 1),   # overlaps lens
    (dict(K=None), 1), (dict(V=0x500002), 3), (dict(nb=16), 4), (dict(rows=7), 2),
])
def test_append_is_checked(lib, kw, status):
    a = dict(K=0x400000, V=0x500000, off=None, rows=4, max_rows=1, lens_out=0x340000, ws=0x900000, nb=256)
    a.update(kw)
    c = _cache()
    assert lib.bdlm_cache_append(a["K"], a["V"], ctypes.cast(ctypes.pointer(c), ctypes.c_void_p), a["off"], a["rows"],
                                 a["max_rows"], a["lens_out"], a["ws"], a["nb"], None) == status, m.bdlm_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(Q=None), 1), (dict(LSE=None), 1), (dict(W=0x700008), 3), (dict(Hq=5), 2), (dict(nb=0), 4),
])
def test_weights_is_checked(lib, kw, status):
    a = dict(Q=0x400000, LSE=0x500000, Hq=4, W=0x700000, nb=256)
    a.update(kw)
    c = _cache()
    assert lib.bdlm_cache_weights(a["Q"], a["LSE"], ctypes.cast(ctypes.pointer(c), ctypes.c_void_p), None, 4, 1,
                                  a["Hq"], 0.125, a["W"], 0x900000, a["nb"], None) == status, m.bdlm_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(keep=0), 2), (dict(sinks=-1), 2), (dict(recent=-1), 2), (dict(sinks=60, recent=5), 2),
    (dict(Wout=0x700000), 1), (dict(Wout=0x700000 + 16), 1),      # overlaps weights
    (dict(dst=0x320000), 1),                                      # the cache's own table
    (dict(lens=0x330004), 1), (dict(W=None), 1), (dict(lens=None), 1), (dict(nb=256), 4),  # room for kept is missing
])
def test_evict_is_checked(lib, kw, status):
    a = dict(W=0x700000, dst=0x350000, keep=64, sinks=4, recent=8, lens=0x340000, Wout=0x800000, kept=None, nb=1 << 20)
    a.update(kw)
    c = _cache()
    assert lib.bdlm_cache_evict(ctypes.cast(ctypes.pointer(c), ctypes.c_void_p), a["W"], a["dst"], a["keep"],
                                a["sinks"], a["recent"], a["lens"], a["Wout"], a["kept"], 0x900000, a["nb"],
                                None) == status, m.bdlm_last_error()


def test_workspace_size(lib):
    size = m.bdlm_workspace_size_cache
    assert size(4, 4, 2, 96, 1) == 0 and size(0, 4, 2, 64, 1) == 0 and size(4, 3, 2, 64, 1) == 0
    assert size(4, 4, 2, 64, 0) == 256 and size(4, 4, 2, 64, -1) == 0
    assert 256 < size(4, 4, 2, 64, 1) < size(4, 4, 2, 64, 200)
    assert size(4, 4, 2, 64, 1, keep=1 << 24) >= 256 + 4 * 2 * (1 << 24) * 4


def test_handle_refuses_host_tensors_and_reassignment(lib):
    f8 = torch.zeros((4, 2, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc, tab, lens = torch.ones(4, 2), torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        m.BdlmCache(f8, f8, sc, sc, tab, lens)
    with pytest.raises(ValueError):
        m.BdlmCache(f8[0], f8, sc, sc, tab, lens)


def test_workspace_views_are_refused():
    """A view with more elements than memory, or with gaps, would be overrun."""
    import types
    cache = types.SimpleNamespace(device=torch.device("cpu"))
    ws = torch.zeros(512, dtype=torch.uint8)
    assert m._cache_workspace(cache, ws, [], 256) is ws
    for bad in (ws[:1].expand(512), ws[::2], ws.view(16, 32).t()):
        with pytest.raises(ValueError, match="contiguous"):
            m._cache_workspace(cache, bad, [], 256)


@pytest.mark.skipif(torch.cuda.is_available(), reason="host-only check of the no-device path")
def test_valid_calls_without_a_device_report_an_error(lib):
    assert _attn(lib) in (5, 6)
