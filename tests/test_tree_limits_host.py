"""Host checks of the calls on drafted trees at the ends of the arguments' ranges (CPU)."""
from __future__ import annotations

import pytest

import structured_mask_attention_gb300 as m
from tests.test_cache_host import lib  # noqa: F401
from tests.test_tree_host import _verify

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("kw", [dict(sp=1 << 40), dict(sq=1 << 40), dict(sp=1 << 40, q=None), dict(sp=1 << 33, sq=1 << 33)])
def test_probabilities_past_64_bit_offsets_are_refused(lib, kw):
    """rows times a stride: bytes that no 64-bit number holds overlap nothing and everything."""
    assert _verify(lib, rows=1 << 30, off=0x340000, **kw) == 2, m.bdlm_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="host-only check of the no-device path")
def test_long_strides_of_few_rows_are_fine(lib):
    assert _verify(lib, sp=1 << 40, sq=1 << 40, p=1 << 50, q=1 << 55) in (5, 6)
