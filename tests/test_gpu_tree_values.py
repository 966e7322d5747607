"""Attention of drafted trees whose own values are of very unlike sizes, on the GPU against 64
bits: what a row does not see does not touch its result, whatever it holds.

Tolerances: check_attn of test_gpu_cache.py.  A weight meets its value off by 2^-11 (2^-22 with fp32 outputs) of
itself and 2^-29 of the largest that the row sees; a row's values are of one size here, so that what is 2^-29 of
the largest is far below the first of check_attn's terms.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

from structured_mask_attention_gb300.inputs import bf16_round
from tests.test_gpu_cache import check_attn, lib  # noqa: F401
from tests.test_gpu_tree_tiles import attend, batch
from tests.tree_plain import plain_attn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

MAX = 2.0 ** 127 * (2 - 2.0 ** -7)  # bf16's largest value
# heads of a group, rows, KV heads (many: a CTA has whole sequences): 16 and 32 columns, split, pairs, several tiles of
# 128, several of 256
SHAPES = [(2, [5, 3], 1), (2, [16, 11], 16), (2, [40, 20], 1), (2, [64, 50], 48), (2, [128, 100], 1), (2, [120, 70], 48),
          (2, [150, 130], 24), (1, [300, 257], 24), (2, [300, 40], 1)]
TYPES = [(64, torch.bfloat16), (64, torch.float32), (128, torch.bfloat16), (128, torch.float32)]


def check(m, x, sees, ref, d, o_dtype):
    check_attn(*attend(m, *x, sees, o_dtype), ref, d, o_dtype == torch.bfloat16)


def random_bits(rows, seed):
    return [np.random.default_rng(seed + n).random((n, n)) < 0.5 for n in rows]


@pytest.mark.parametrize("g,rows,Hkv", SHAPES)
@pytest.mark.parametrize("value", [1e4, 1e30, -MAX])
@pytest.mark.parametrize("d,o_dtype", TYPES)
@pytest.mark.parametrize("lens", [[0, 210], [600, 0]])
def test_hidden_rows_hold_large_values(lib, g, rows, Hkv, value, d, o_dtype, lens):
    """A third of the own rows is seen by none and holds large finite keys and values."""
    x = batch(lens, rows, g, Hkv, d, 16, 9)
    sees = random_bits(rows, 1)
    for see in sees:
        see[:, 1::3] = False
    ref = plain_attn(torch, *(x[i] for i in (0, 2, 3, 4)), sees, x[1], 1 / math.sqrt(d))
    for s, n in enumerate(rows):
        for t in x[3:]:
            t[x[1][s]:x[1][s + 1]][1::3] = value
    check(lib, x, sees, ref, d, o_dtype)


@pytest.mark.parametrize("g,rows,Hkv", SHAPES)
@pytest.mark.parametrize("value", [1e6, 1e30])
@pytest.mark.parametrize("d,o_dtype", TYPES)
def test_rows_that_see_a_large_value_and_rows_that_do_not(lib, g, rows, Hkv, value, d, o_dtype):
    x = batch([300, 0], rows, g, Hkv, d, 32, 3)
    sees = random_bits(rows, 2)
    V = x[4]
    for s, n in enumerate(rows):
        at = x[1][s] + n // 2
        V[at] = bf16_round(np.float32(value) * np.sign(V[at]))
    ref = plain_attn(torch, *(x[i] for i in (0, 2, 3, 4)), sees, x[1], 1 / math.sqrt(d))
    check(lib, x, sees, ref, d, o_dtype)


@pytest.mark.parametrize("g,rows,Hkv", SHAPES[2:])
@pytest.mark.parametrize("value,rest", [(2.0 ** 120, 1.0), (2.0 ** 120, 2.0 ** 80), (2.0 ** 125, 0.0), (1.0, 2.0 ** -60)])
@pytest.mark.parametrize("d,o_dtype", TYPES)
def test_values_at_the_ends_of_the_range(lib, g, rows, Hkv, value, rest, d, o_dtype):
    """Every fifth row holds values of 2^120 (of 1), which every other row sees, the rest of 1, 2^80 or 0 (of 2^-60)."""
    x = batch([300, 0], rows, g, Hkv, d, 32, 6)
    size = np.where(np.arange(sum(rows)) % 5 == 2, value, rest)
    x[4][:] = bf16_round((np.clip(np.abs(x[4]), 0.25, 4) * np.sign(x[4]) * size[:, None, None]).astype(np.float32))
    sees = random_bits(rows, 5)
    for see in sees:
        see[1::2, 2::5] = False
    ref = plain_attn(torch, *(x[i] for i in (0, 2, 3, 4)), sees, x[1], 1 / math.sqrt(d))
    check(lib, x, sees, ref, d, o_dtype)


@pytest.mark.parametrize("g,rows,Hkv", SHAPES)
@pytest.mark.parametrize("d,o_dtype", TYPES)
@pytest.mark.parametrize("cached", [False, True])
def test_rows_that_see_themselves_alone(lib, g, rows, Hkv, d, o_dtype, cached):
    """Values from 2^-40 to 2^40, each seen by its own row, beside cached ones of about 2^-45."""
    x = batch([300, 40] if cached else [0, 0], rows, g, Hkv, d, 32, 4)
    x[0]["vs"] *= np.float32(2.0 ** -45)
    size = 2.0 ** ((np.arange(sum(rows)) * 7 % 81) - 40)
    x[4][:] = bf16_round((x[4] * size[:, None, None]).astype(np.float32))
    sees = [np.eye(n, dtype=bool) for n in rows]
    ref = plain_attn(torch, *(x[i] for i in (0, 2, 3, 4)), sees, x[1], 1 / math.sqrt(d))
    check(lib, x, sees, ref, d, o_dtype)


@pytest.mark.parametrize("g,rows,Hkv", SHAPES)
@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** 20])
@pytest.mark.parametrize("d,o_dtype", TYPES)
@pytest.mark.parametrize("cached", [False, True])
def test_values_of_zero_count_in_the_row_sum(lib, g, rows, Hkv, size, d, o_dtype, cached):
    """Every other own row has values of zero and takes its part of the weights all the same."""
    x = batch([300, 40] if cached else [0, 0], rows, g, Hkv, d, 32, 5)
    x[4][:] = bf16_round(x[4] * np.float32(size))
    x[4][1::2] = 0
    sees = random_bits(rows, 3)
    ref = plain_attn(torch, *(x[i] for i in (0, 2, 3, 4)), sees, x[1], 1 / math.sqrt(d))
    check(lib, x, sees, ref, d, o_dtype)


@pytest.mark.parametrize("g,rows,Hkv", SHAPES)
@pytest.mark.parametrize("d,o_dtype", TYPES)
@pytest.mark.parametrize("value", [math.nan, 1e30])
def test_cached_values_far_below_own_ones_keep_their_weights(lib, g, rows, Hkv, d, o_dtype, value):
    """Cached values of 2^-70, own ones of 2^10, beside hidden rows of NaN or 1e30: the scales that a row sees differ by
    less than 2^100, and the cached keys' weights, most of the sum, count in it."""
    x = batch([1700, 300], rows, g, Hkv, d, 64, 8)
    x[0]["vs"] *= np.float32(2.0 ** -70)
    x[4][:] *= np.float32(2.0 ** 10)
    sees = [see | np.eye(len(see), dtype=bool) for see in random_bits(rows, 7)]
    for see in sees:
        see[:, 1::3] = False
    ref = plain_attn(torch, *(x[i] for i in (0, 2, 3, 4)), sees, x[1], 1 / math.sqrt(d))
    for s in range(2):
        x[4][x[1][s]:x[1][s + 1]][1::3] = value
    check(lib, x, sees, ref, d, o_dtype)
