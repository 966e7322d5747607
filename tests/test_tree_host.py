"""Host checks of the calls on drafted trees: argument validation before anything
reaches a device (CPU)."""
from __future__ import annotations

import ctypes

import pytest

import structured_mask_attention_gb300 as m
from tests.test_cache_host import _cache, lib  # noqa: F401

torch = pytest.importorskip("torch")

REF = lambda c: ctypes.cast(ctypes.pointer(c), ctypes.c_void_p)


def _mask(lib, par=0x400000, off=None, rows=8, max_rows=2, vis=0x500000, words=1, pos=0x600000, ws=0x900000, nb=256):
    return lib.bdlm_tree_mask(par, REF(_cache()), off, rows, max_rows, vis, words, pos, ws, nb, None)


def _tree(lib, Q=0x400000, K=0x500000, V=0x600000, vis=0xa00000, words=1, off=None, rows=4, max_rows=1, Hq=4, scale=0.125,
          O=0x700000, dt=0, LSE=0x800000, ws=0x900000, nb=1 << 30):
    return lib.bdlm_attn_tree(Q, K, V, vis, words, REF(_cache()), off, rows, max_rows, Hq, scale, O, dt, LSE, ws, nb, None)


def _verify(lib, par=0x100000, tok=0x110000, p=0x200000, q=0x300000, dt=1, V=100, sp=100, sq=100, u=0x120000, s=0x130000,
            n=4, off=None, rows=8, max_rows=2, path=0x140000, max_path=2, acc=0x150000, nxt=0x160000, ws=0x900000, nb=256):
    return lib.bdlm_tree_verify(par, tok, p, q, dt, V, sp, sq, u, s, n, off, rows, max_rows, path, max_path, acc, nxt, ws, nb,
                                None)


def _commit(lib, K=0x400000, V=0x500000, path=0x600000, max_path=3, acc=0x610000, off=None, rows=8, max_rows=2,
            out=0x340000, ws=0x900000, nb=256):
    return lib.bdlm_cache_commit(K, V, REF(_cache()), path, max_path, acc, off, rows, max_rows, out, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(words=0), 2), (dict(words=(1 << 19) + 1), 2), (dict(max_rows=33, rows=132), 2), (dict(max_rows=4097, rows=16388), 2),
    (dict(rows=7), 2), (dict(par=None), 1), (dict(vis=None), 1), (dict(pos=None), 1), (dict(pos=0x600002), 3),
    (dict(ws=None), 4), (dict(nb=255), 4), (dict(off=0x340002), 3),
    (dict(vis=0x400000 + 28), 1), (dict(pos=0x400000 - 28), 1), (dict(pos=0x500000 + 4), 1),       # overlaps
    (dict(vis=0x330000), 1), (dict(pos=0x330004), 1), (dict(vis=0x340010, off=0x340000, words=1), 1),
])
def test_mask_is_checked(lib, kw, status):
    assert _mask(lib, **kw) == status, m.bdlm_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=3), 2), (dict(scale=0.0), 1), (dict(dt=2), 1), (dict(K=None), 1), (dict(V=None), 1), (dict(K=None, V=None), 1),
    (dict(Q=None), 1), (dict(vis=None), 1), (dict(vis=0xa00002), 3), (dict(words=0), 2), (dict(words=(1 << 19) + 1), 2),
    (dict(max_rows=33, rows=132), 2), (dict(max_rows=65, rows=260, words=2), 2), (dict(ws=None), 4), (dict(nb=256), 4),
    (dict(rows=5), 2), (dict(O=0x400000), 1), (dict(O=0xa00000 - 2048 + 16), 1), (dict(LSE=0xa00000 + 12), 1),
])
def test_attn_is_checked(lib, kw, status):
    assert _tree(lib, **kw) == status, m.bdlm_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), 2), (dict(n=65536), 2), (dict(max_rows=4097, rows=16388), 2), (dict(rows=9), 2), (dict(dt=2), 1),
    (dict(V=0), 2), (dict(V=(1 << 30) + 1, sp=1 << 31, sq=1 << 31), 2), (dict(sp=99), 2), (dict(sq=99), 2),
    (dict(sp=(1 << 40) + 1), 2), (dict(max_path=0), 2), (dict(max_path=(1 << 24) + 1), 2),
    (dict(par=None), 1), (dict(tok=None), 1), (dict(p=None), 1), (dict(u=None), 1), (dict(s=None), 1), (dict(path=None), 1),
    (dict(acc=None), 1), (dict(nxt=None), 1), (dict(p=0x200002), 3), (dict(q=0x300002), 3), (dict(p=0x200001, dt=0), 3),
    (dict(ws=None), 4), (dict(nb=255), 4), (dict(ws=0x900008), 3),
    (dict(path=0x100000 + 28), 1), (dict(acc=0x200000 + 3196), 1), (dict(nxt=0x300000 + 3196), 1), (dict(acc=0x130000), 1),
    (dict(acc=0x140000 + 28), 1), (dict(nxt=0x150000), 1), (dict(nxt=0x120000 + 28), 1), (dict(path=0x340010, off=0x340000), 1),
])
def test_verify_is_checked(lib, kw, status):
    assert _verify(lib, **kw) == status, m.bdlm_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(K=None), 1), (dict(V=0x500002), 3), (dict(path=None), 1), (dict(acc=None), 1), (dict(max_path=0), 2),
    (dict(max_path=(1 << 24) + 1), 2), (dict(rows=9), 2), (dict(nb=16), 4), (dict(acc=0x610002), 3),
    (dict(out=0x330000), 1), (dict(out=0x600000 + 44), 1), (dict(out=0x610008), 1), (dict(out=0x340004, off=0x340000), 1),
])
def test_commit_is_checked(lib, kw, status):
    assert _commit(lib, **kw) == status, m.bdlm_last_error()


def test_null_cache(lib):
    assert lib.bdlm_tree_mask(0x400000, None, None, 4, 1, 0x500000, 1, 0x600000, 0x900000, 256, None) == 1
    assert lib.bdlm_cache_commit(1 << 20, 1 << 20, None, 1 << 21, 1, 1 << 22, None, 4, 1, None, 1 << 23, 256, None) == 1


def test_no_rows_is_no_work(lib):
    assert _mask(lib, off=0x340000, rows=0, par=None, vis=None, pos=None) == 0
    assert _tree(lib, off=0x340000, rows=0, Q=None, K=None, V=None, vis=None) == 0


def test_workspace_size(lib):
    size = m.bdlm_workspace_size_verify
    assert size(4, 2, 100) >= 256 and size(0, 2, 100) == 0 and size(4, 0, 100) == 0 and size(4, 4097, 100) == 0
    assert size(4, 2, 0) == 0 and size(65536, 2, 100) == 0
    with pytest.raises(ValueError):
        m.bdlm_verify_workspace(0, 1, 1)


def test_python_refuses_host_tensors_and_odd_layouts(lib):
    i, f, p = torch.zeros(4, dtype=torch.int32), torch.zeros(4), torch.zeros(4, 9)
    for bad in (p, p.double(), p.t(), p[:, ::2]):
        with pytest.raises(ValueError):
            m.bdlm_tree_verify(i, i, bad, None, f, f[:1])
    import types
    cache = types.SimpleNamespace(device=torch.device("cpu"), Hkv=1, d=64, n_seqs=1)
    Q = torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="both"):
        m.bdlm_attn_tree(Q, None, Q, i[:, None], cache)
    with pytest.raises(ValueError, match="visible"):
        m.bdlm_attn_tree(Q, Q, Q, i, cache)
    with pytest.raises(ValueError, match="path"):
        m.bdlm_cache_commit(cache, Q, Q, i, i[:1])


@pytest.mark.skipif(torch.cuda.is_available(), reason="host-only check of the no-device path")
def test_valid_calls_without_a_device_report_an_error(lib):
    for call in (_mask, _tree, _verify, _commit):
        assert call(lib) in (5, 6), m.bdlm_last_error()
    assert _verify(lib, q=None, sq=0) in (5, 6)
