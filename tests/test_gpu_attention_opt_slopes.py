"""Distance slopes below zero, where far keys count more: the weights that a
query past the sequence's end would have overflow (exp of |slope| times a
distance above 88.7), and nothing of them may reach the gradients.  Tolerances
are the oracle's."""
import numpy as np
import pytest
import torch

import oracle.attention_opt as O

from gpu_util import to_f64
from test_gpu_attention_opt import Problem

pytestmark = pytest.mark.gpu


def with_slopes(kind, b, s, d, cap, slopes):
    p = Problem(kind, b, s, len(slopes), d, cap, True)
    p.slopes = slopes
    p.sl.copy_(torch.tensor(slopes))
    return p


@pytest.mark.parametrize("s", [200, 430, 1037])
@pytest.mark.parametrize("kind", ["causal", "whole"])
@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("d", [64, 128])
def test_negative_slopes_at_ragged_lengths(s, kind, cap, d):
    with_slopes(kind, 1, s, d, cap, [-1.0, -0.25, -0.5]).check()


@pytest.mark.parametrize("kind", ["documents", "prefix", "any"])
def test_negative_slopes_over_sequences_and_masks(kind):
    with_slopes(kind, 2, 333, 64, 0.0, [-2.0, 0.5]).check()


@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_steep_negative_slopes(cap):
    """Rows of nearly one key.  dz is then the small difference of dP and delta,
    whose own rounding (of the stored O) the element-wise tolerance counts and a
    norm in steps of dz would not."""
    p = with_slopes("causal", 1, 600, 64, cap, [-4.0, -30.0])
    qkv, dout = to_f64(p.qkv), to_f64(p.dout)
    o, _, tol, _ = O.attention_forward(qkv, p.lo, p.hi, p.H, p.d, p.slopes, cap)
    assert (np.abs(p.forward()[0] - o) <= tol).all()
    ref, tol, _ = O.attention_backward(qkv, dout, p.lo, p.hi, p.H, p.d, p.slopes, cap)
    for tiles in (False, True):
        assert (np.abs(p.backward(tiles) - ref) <= tol).all()
