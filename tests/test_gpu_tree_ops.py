"""Verification of drafted trees whose probabilities add up to more than a distribution's, and commits on
lengths out of range, on the GPU against the fp64 oracle.  Everything compared is whole numbers: equal."""
from __future__ import annotations

import numpy as np
import pytest

from tests.cache_util import device_cache, host_codes, make_cache, make_rows
from tests.parity_util import to_dev
from tests.test_gpu_cache import lib  # noqa: F401
from tests.test_gpu_tree import DEV, run_verify

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ones", [2, 3])
@pytest.mark.parametrize("V", [4, 7, 61, 1003])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_rows_that_sum_to_two_and_more(lib, ones, V, drawn, dtype):
    """p is 1 at two or three tokens side by side (in one thread's hands) and 0.75 more at others, 3.75 at most."""
    def spoil(parents, tokens, target, draft, us, s):
        target *= np.float32(0.75)
        first = V // 3
        target[:, first:first + ones] = 1
        rest = np.ones(V, bool)
        rest[first:first + ones] = False
        target[:, rest] *= np.float32(0.75) / target[:, rest].sum(1, keepdims=True)
        tokens[::3] = V - 1
        if dtype == torch.bfloat16:
            target[:] = torch.from_numpy(target).to(dtype).float().numpy()
        s[:] = (np.arange(len(s)) + 0.5) / len(s)
    for seed in range(3):
        ws, got = run_verify(lib, [9] * 40, 3, V, drawn, dtype, seed=seed, spoil=spoil)
        lib.bdlm_sync_status(ws)


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_every_token_of_large_sums_can_be_drawn(lib, drawn):
    """Four tokens of p = 1, 1, 1, 0.5: sample in sevenths of the sum names each in its turn."""
    p = torch.tensor([[1.0, 1.0, 1.0, 0.5]], device="cuda").repeat(7, 1)
    q = torch.zeros_like(p) if drawn else None
    i = torch.zeros(7, dtype=torch.int32, device="cuda")
    s = (torch.arange(7, device="cuda") + 0.5) / 7
    path, acc, tok = lib.bdlm_tree_verify(i - 1, i, p, q, s, s)
    assert acc.tolist() == [1] * 7 and tok.tolist() == [0, 0, 1, 1, 2, 2, 3]


@pytest.mark.parametrize("lens", [[-1, 9], [9, -2 ** 31], [9, 49], [2 ** 31 - 1, 0]])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 128)])
def test_commit_treats_lengths_out_of_range_as_the_append_does(lib, lens, d, page):
    """A negative length counts as 0, one behind the page table as the table's end; the call reports it."""
    m = lib
    c, _ = make_cache([9, 9], 40, 2, d, page, seed=5)
    K, V = (to_dev(make_rows(10, 2, d, s), torch) for s in (1, 2))
    made = []
    for commit in (False, True):
        cache = device_cache(m, torch, c)
        cache.lens.copy_(torch.tensor([min(x, 2 ** 31 - 1) if x != 49 else -(-40 // page) * page + 1 for x in lens],
                                      dtype=torch.int32))
        ws = m.bdlm_cache_workspace(cache)
        if commit:
            path = DEV(np.tile(np.arange(5, dtype=np.int32), (2, 1)))
            out = m.bdlm_cache_commit(cache, K, V, path, DEV(np.asarray([5, 5], np.int32)), workspace=ws)
        else:
            out = m.bdlm_cache_append(cache, K, V, workspace=ws)
        with pytest.raises(m.BdlmError, match="length"):
            m.bdlm_sync_status(ws)
        made.append([out.cpu().numpy()] + [host_codes(getattr(cache, w + "8")) for w in "kv"]
                    + [getattr(cache, w + "_scale").cpu().numpy() for w in "kv"])
    for a, b in zip(*made):
        np.testing.assert_array_equal(a, b)
