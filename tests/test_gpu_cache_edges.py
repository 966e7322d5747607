"""The 8-bit cache's calls where their number formats end (GPU): a dominant
key, blocks of zeros, tiny queries, channels of unlike size, sequences without
new rows; and what the status words say.  Tolerances as in test_gpu_cache.py,
with the floors that the header gives added where a test reaches them."""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle.cache_oracle as co
from tests.cache_util import device_cache, host_codes, make_cache, make_rows
from tests.parity_util import to_dev
from tests.test_gpu_cache import lib  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


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
