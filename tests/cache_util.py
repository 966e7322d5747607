"""Small caches for the tests of the 8-bit cache: the same arrays on the host
(for the oracle) and on the device."""
from __future__ import annotations

import numpy as np

from structured_mask_attention_gb300.inputs import bf16_round


def offsets_of(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


def make_cache(lens, capacity, Hkv, d, page, seed, sets=1, stale=127):
    """A host cache with sequences of the given lengths on scattered pages, room for ``capacity`` tokens each (and
    ``sets`` - 1 more tables of spare pages).  Every code behind a sequence's length and on unused pages is
    ``stale`` (127: NaN), every scale of an unused page NaN: none of it may be read into a result."""
    rng = np.random.default_rng(seed)
    n, mp = len(lens), -(-capacity // page)
    n_pages = sets * n * mp + 2
    ids = rng.permutation(n_pages)[: sets * n * mp].astype(np.int32).reshape(sets, n, mp)
    c = {"table": np.ascontiguousarray(ids[0]), "lens": np.asarray(lens, np.int32)}
    for w in ("k", "v"):
        codes = np.full((n_pages, Hkv, page, d), stale, np.uint8)
        scales = np.full((n_pages, Hkv), np.nan, np.float32)
        for s, L in enumerate(lens):
            for j in range(-(-int(L) // page)):
                m, p = min(page, int(L) - j * page), ids[0, s, j]
                # magnitudes up to 448, all signs and exponents; scales such that values are about N(0, 1)
                x = np.clip(rng.standard_normal((Hkv, m, d)) * 110.0, -448, 448)
                from oracle.cache_oracle import encode
                codes[p, :, :m] = encode(x)
                scales[p] = 2.0 ** (rng.integers(-1, 2, Hkv) - 7)
        c[w + "8"], c[w + "s"] = codes, scales
    return c, [np.ascontiguousarray(x) for x in ids[1:]]


def make_rows(T, H, d, seed):
    return bf16_round(np.random.default_rng(seed).standard_normal((T, H, d), dtype=np.float32))


def device_cache(m, torch, c, device="cuda"):
    """A BdlmCache over copies of the host cache's arrays."""
    f8 = lambda x: torch.from_numpy(x.copy()).to(device).view(torch.float8_e4m3fn)
    t = lambda x: torch.from_numpy(x.copy()).to(device)
    return m.BdlmCache(f8(c["k8"]), f8(c["v8"]), t(c["ks"]), t(c["vs"]), t(c["table"]), t(c["lens"]))


def host_codes(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()
