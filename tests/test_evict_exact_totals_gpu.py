"""pa_pool_evict's totals: the exact sum over the heads rounded to fp32, also where fp32 sums with their errors carried
along are not enough: borders between two numbers, sums that cancel or pass fp32's range on the way."""
from fractions import Fraction

import numpy as np
import pytest

from tests import evict_model
from tests.test_pool_evict_gpu import append, both, evict, score

pytestmark = pytest.mark.gpu


def rounded(column):
    """The exact sum of a column, rounded once to fp32, halves to even."""
    if np.isnan(column).any() or (np.isposinf(column).any() and np.isneginf(column).any()):
        return np.float32(np.nan)
    if np.isinf(column).any():
        return column[np.isinf(column)][0]
    total = sum(map(Fraction, column.tolist()))
    size, step = abs(total), Fraction(2) ** -149
    while size >= step * 2 ** 24:
        step *= 2
    whole = size // step
    rest = size / step - whole
    whole += rest > Fraction(1, 2) or (rest == Fraction(1, 2) and whole % 2 == 1)
    value = whole * step
    return np.float32(np.copysign(np.inf if value >= 2 ** 128 else float(value), -1 if total < 0 else 1))


@pytest.fixture(autouse=True)
def model_rounds_once(monkeypatch):
    """(The model's own sum is rounded to 64 bits before it is rounded to 32.)"""
    monkeypatch.setattr(evict_model, "totals", lambda scores: np.array([rounded(x) for x in scores.T], np.float32))


def totals(columns, hkv, lens, budget, apart=False, width=8, bs=16):
    """Rows of these lengths whose tokens' scores are columns drawn in turn; what stays is as the model says."""
    dims, pool, model = both("bf16", 1, width * len(lens) + 3, bs, hkv, 64, len(lens) + 1, width)
    append(dims, pool, model, list(range(len(lens))), lens)
    s = score(pool, model, hkv, 1)
    r = np.random.default_rng(7)
    for row, n in zip(s, lens):
        row[:, :n] = columns[r.integers(0, len(columns), n)].T
    assert evict(dims, pool, model, list(range(len(lens))), s, budget, 0, 0, apart) is not None


HARD = [
    [1, 2.0 ** -24, 2.0 ** -48], [1, 2.0 ** -24, 0], [1, 2.0 ** -24, 2.0 ** -100], [1, 2.0 ** -24, 2.0 ** -149],
    [2.0 ** -149, 2.0 ** -24, 1], [1 + 2.0 ** -23, 2.0 ** -24, 0], [1 + 2.0 ** -23, 2.0 ** -24, -2.0 ** -120],
    [1, 2.0 ** -25, 2.0 ** -25], [1, -2.0 ** -25, 0], [1, -2.0 ** -25, -2.0 ** -60], [1, 0, 0], [1 - 2.0 ** -24, 0, 0],
    [1e30, -1e30, 1], [1e30, 1, -1e30], [3e38, 3e38, -3e38], [3e38, 3e38, 3e38], [-3e38, -3e38, 3e38], [3e38, -3e38, 1],
    [np.inf, 1, 1], [np.inf, -np.inf, 1], [-np.inf, 1, 3e38], [np.nan, 1, 1], [0.0, -0.0, 0.0], [-0.0, -0.0, -0.0],
    [2.0 ** -149, -2.0 ** -149, 0], [2.0 ** -126, -2.0 ** -149, 0], [2.0 ** 127, 2.0 ** 127 * (1 - 2.0 ** -24), 2.0 ** 102],
    [2.0 ** 127, 2.0 ** 127 * (1 - 2.0 ** -24), 2.0 ** 103], [2.0 ** 24, 1, 2.0 ** -149], [2.0 ** 24, 1, 0], [2.0 ** 24, 2, 0],
]


@pytest.mark.parametrize("budget", [1, 10, 50, 100])
def test_borders_and_cancelled_sums(budget):
    totals(np.array(HARD, np.float32), 3, [120, 33, 101], budget)


@pytest.mark.parametrize("hkv", [1, 2, 4, 5, 8, 16, 33])
def test_sums_near_borders(hkv):
    """Random columns of few powers of two, so that many sums fall on or next to the middle of two fp32 numbers."""
    r = np.random.default_rng(hkv)
    e = r.choice([0, -1, -23, -24, -25, -47, -48, -49, -72, -100], (60, hkv))
    x = np.where(r.random((60, hkv)) < 0.7, 2.0 ** e, 0)
    x[:30] *= r.choice([1, -1], (30, hkv))
    x[:, 0] = 1
    totals(x.astype(np.float32), hkv, [128, 100], 40, apart=hkv % 2 == 1)


def test_two_tokens_apart_by_a_sum_next_to_a_border():
    """1 + 2^-24 + 2^-48 is 1 + 2^-23 in fp32, more than 1, though its index is the higher."""
    x = np.zeros((3, 40), np.float32)
    x[0] = 1
    x[1, 30], x[2, 30] = 2.0 ** -24, 2.0 ** -48
    assert evict_model.choose(x, 40, 1, 0, 0).tolist() == [30]
    dims, pool, model = both("bf16", 1, 8, 16, 3, 64, 2, 4)
    append(dims, pool, model, [0], [40])
    s = score(pool, model, 3, 1)
    s[0, :, :40] = x
    kept = evict(dims, pool, model, [0], s, 1, 0, 0)[0]
    assert kept.tolist() == [[30]]


def test_rows_beyond_shared_memory(monkeypatch):
    dims, pool, model = both("bf16", 1, 60, 1024, 3, 64, 2, 57)
    append(dims, pool, model, [1], [50000])
    s = score(pool, model, 3, 1)
    pick = np.random.default_rng(1).integers(0, len(HARD), 50000)
    s[1, :, :50000] = np.array(HARD, np.float32)[pick].T
    of = np.array([rounded(np.array(x, np.float32)) for x in HARD], np.float32)
    monkeypatch.setattr(evict_model, "totals", lambda scores: of[pick])
    assert evict(dims, pool, model, [1], s, 20000, 0, 0) is not None
