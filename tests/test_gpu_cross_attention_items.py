"""Attention to long keys with more items than SMs, heads of 128, forward: the kernel
that keeps one CTA on an SM then walks several items, or takes over unstarted ones,
longest first or in their order, empty ones among them."""
import os
import subprocess
import sys

import pytest
import torch

from megatron_transformer_layer_gb300 import _lib as L

from gpu_util import check_status
from test_gpu_attention_opt_debug import TESTS, digest
from test_gpu_cross_attention import Problem
from test_gpu_cross_attention_streams import Attention

pytestmark = pytest.mark.gpu

LENS = [1030, 0, 1, 1024, 0, 0, 129, 961, 256, 0, 1030, 257]


def offsets(lens):
    out = [7]
    for n in lens:
        out.append(out[-1] + n)
    return out


def padded():
    """Lengths that differ, some 0: sorted, and taken over."""
    return Problem(24, 24 * 5, 24 * 1030, 8, 8, 128, kv_lens=LENS * 2)


def equal(n, heads, sq, sk):
    """Nothing to sort: a fixed walk, and taken over where there are many."""
    return Problem(n, n * sq, n * sk, heads, heads, 128)


def packed(n):
    """More sequences than are sorted, most of them without keys, a few without queries."""
    k = [0 if i % 5 else LENS[i // 5 % len(LENS)] for i in range(n)]
    q = [i % 4 for i in range(n)]
    ko, qo = offsets(k), offsets(q)
    return Problem(n, qo[-1] + 3, ko[-1] + 40, 4, 4, 128, q_offsets=qo, kv_offsets=ko, max_q=3,
                   max_kv=1030)


def grouped():
    """Two heads to a key head, and blocks of which whole warps have no query."""
    lens = [70, 3, 0, 64, 65, 17, 33, 1, 70, 48]
    return Problem(30, 30 * 70, 30 * 1000, 12, 6, 128, q_lens=lens * 3,
                   kv_lens=[min(n, 1000) for n in (LENS * 3)[:30]], wide=128)


CASES = [padded, lambda: equal(2, 40, 300, 1000), lambda: equal(4, 64, 260, 970),
         lambda: packed(80), lambda: packed(170), grouped]


@pytest.mark.parametrize("case", CASES)
def test_against_the_oracle(case):
    case().check_forward()


def test_gradients():
    grouped().check()


def test_same_bits_again():
    for case in (padded, CASES[4]):
        p = case()
        p.forward()
        o, lse = p.o_all.clone(), p.lse.clone()
        for _ in range(5):
            p.forward()
            assert torch.equal(p.o_all, o) and torch.equal(p.lse, lse)


def test_two_streams_at_once():
    a, b = (Attention(24, 5, 1030, 8, 8, 128, LENS * 2, seed=s) for s in (0, 50))
    want = [p.alone() for p in (a, b)]
    sides = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for side, p in zip(sides, (a, b)):
            assert p.step(side) == [0, 0]
    torch.cuda.synchronize()
    for p, w in zip((a, b), want):
        assert all(torch.equal(x, y) for x, y in zip(p.outputs(), w))
        check_status(p.st)


def results():
    out = []
    for case in (padded, CASES[3], CASES[4], grouped):
        p = case()
        p.forward()  # (checks the status)
        out.append(digest(p.o_all, p.lse))
    return out


def test_debug_build_is_clean_and_matches_release():
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "from megatron_transformer_layer_gb300 import _lib as L\n"
            "assert L.LIB_PATH.endswith('_debug.so')\n"
            "from test_gpu_cross_attention_items import results\n"
            "for r in results(): print(r)\n") % (os.path.dirname(TESTS), TESTS)
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600,
                         env=dict(os.environ, MC_LAYER_DEBUG="1"))
    assert out.returncode == 0, out.stderr[-2000:]
    assert not L.LIB_PATH.endswith("_debug.so")
    assert out.stdout.split() == results()
