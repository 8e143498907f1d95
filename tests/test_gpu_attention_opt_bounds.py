"""Interval bounds anywhere in 32 bits: what lies outside the sequence is cut to
it, so the lowest and the highest integer mean "no limit" or "nothing"."""
import numpy as np
import pytest

from megatron_transformer_layer_gb300 import _lib as L

from gpu_util import check_status, status
from test_gpu_attention_opt import Problem, i32, random_intervals, table_lists
import oracle.attention_opt as O

pytestmark = pytest.mark.gpu

LOW, HIGH = -(2 ** 31), 2 ** 31 - 1


def extreme_intervals(b, s):
    """Intervals with no order in which 32-bit limits stand for everything
    outside the sequence, and rows that those leave empty."""
    lo, hi = random_intervals(b, s, 3 * s)
    lo, hi = np.where(lo <= 0, LOW, lo), np.where(hi >= s, HIGH, hi)
    t = np.arange(s)
    hi = np.where(t % 7 == 3, HIGH, hi)
    lo = np.where(t % 5 == 1, LOW, lo)
    hi = np.where(t % 11 == 4, LOW, hi)     # empty rows
    lo = np.where(t % 13 == 6, HIGH, lo)
    return lo, hi


def problem(b, s, H, d, cap, bias, lo, hi):
    p = Problem("any", b, s, H, d, cap, bias)
    p.lo, p.hi = lo, hi
    p.klo.copy_(i32(lo))
    p.khi.copy_(i32(hi))
    st = status()
    assert L.mc_attention_mask_intervals(b, s, p.klo, p.khi, p.tab, st) == 0
    check_status(st)
    return p


@pytest.mark.parametrize("cap,bias", [(0.0, False), (4.0, False), (0.0, True), (4.0, True)])
@pytest.mark.parametrize("b,s,H,d", [(1, 700, 2, 64), (2, 333, 2, 128)])
def test_bounds_at_the_ends_of_32_bits(b, s, H, d, cap, bias):
    lo, hi = extreme_intervals(b, s)
    p = problem(b, s, H, d, cap, bias, lo, hi)
    assert table_lists(p.tab) == O.tables(lo, hi)
    p.check()


def test_no_limits_see_all():
    """(lowest, highest) in every row is the whole sequence."""
    b, s = 1, 520
    lo, hi = np.full((b, s), LOW), np.full((b, s), HIGH)
    problem(b, s, 2, 64, 0.0, False, lo, hi).check()
