"""Gradients of sequences with few keys: as exact, and the same to the bit, whatever
other sequences the call has and whatever bounds or slots it states for them."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle.cross_attention as O
from megatron_transformer_layer_gb300 import _lib as L

from gpu_util import DEV, check_status, status, to_f64
from test_gpu_attention_opt_debug import TESTS, digest
from test_gpu_cross_attention import Problem

pytestmark = pytest.mark.gpu

LENS = [300, 2, 9, 128, 3, 129, 1, 64]


def offsets(lens):
    return [int(x) for x in np.concatenate([[0], np.cumsum(lens)])]


def backward(p, q_rows, k_rows, **rows):
    """dq, dk, dv of a call over these slices of p's rows, on p's O and lse."""
    q, k = slice(*q_rows), slice(*k_rows)
    nq, nk = q.stop - q.start, k.stop - k.start
    n = rows.pop("n", 1)
    c = L.make_cross_attention(n, nq, nk, p.heads, p.kv_heads, p.d, ld_q=p.q_all.stride(0),
                               ld_kv=p.kv_all.stride(0), ld_o=p.o_all.stride(0), **rows)
    dq_all, dkv_all = torch.zeros_like(p.q_all[q]), torch.zeros_like(p.kv_all[k])
    dq, dk, dv = dq_all[:, : p.a], dkv_all[:, : p.akv], dkv_all[:, p.akv: 2 * p.akv]
    lse = p.lse[:, q].contiguous()
    delta = torch.full_like(lse, float("nan"))
    ws = torch.full((L.mc_attention_backward_cross_ws_bytes(c),), 0xff, dtype=torch.uint8, device=DEV)
    st = status()
    assert L.mc_attention_backward_cross(p.q[q], p.k[k], p.v[k], p.o[q], lse, p.dout[q], dq, dk, dv,
                                         delta, c, ws, ws.numel(), st) == 0
    check_status(st)
    return dq, dk, dv


def problems(d, heads, kv_heads, sq):
    """The lengths in slots of 300 rows, packed with a bound, and packed without one."""
    n, off = len(LENS), offsets(LENS)
    q_off = offsets([sq] * n)
    yield Problem(n, n * sq, n * 300, heads, kv_heads, d, kv_lens=LENS)
    yield Problem(n, n * sq, off[-1], heads, kv_heads, d, q_offsets=q_off, kv_offsets=off, max_q=sq,
                  max_kv=300)
    yield Problem(n, n * sq, off[-1], heads, kv_heads, d, q_offsets=q_off, kv_offsets=off)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,sq", [(4, 4, 140), (6, 2, 33), (8, 1, 1)])
def test_a_short_sequence_beside_long_ones(d, heads, kv_heads, sq):
    for p in problems(d, heads, kv_heads, sq):
        p.check()
        got = p.dq_all[:, : p.a], p.dkv_all[:, : p.akv], p.dkv_all[:, p.akv: 2 * p.akv]
        for (q0, _, nq), (k0, _, nk) in zip(p.q_seq, p.k_seq):
            if nk > 128:
                continue
            alone = backward(p, (q0, q0 + nq), (k0, k0 + nk))
            for name, x, y in zip(("dQ", "dK", "dV"), got, alone):
                at, rows = (q0, nq) if name == "dQ" else (k0, nk)
                assert torch.equal(x[at: at + rows], y), (name, nk)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(4, 4), (6, 2)])
def test_errors_of_short_sequences(d, heads, kv_heads):
    """What the cancellation in dP - delta leaves, sequence by sequence: roundings to
    bf16 of dz and dQ (together below 2^-7 of the 2-norm) beside 2^-16 of the terms'
    size, as where all sequences have few keys."""
    for p in problems(d, heads, kv_heads, 90):
        p.check()
        dq = to_f64(p.dq_all)[:, : p.a]
        ref, _, _ = O.backward(*map(p.clean, (p.q, p.k, p.v, p.dout)), p.q_seq, p.k_seq, heads,
                               kv_heads, d, p.scale)
        for (q0, _, nq), (k0, _, nk) in zip(p.q_seq, p.k_seq):
            if nk > 128:
                continue
            q, k = slice(q0, q0 + nq), slice(k0, k0 + nk)
            size = p.scale * np.linalg.norm(p.clean(p.k)[k], axis=1).max() * \
                np.linalg.norm(p.clean(p.v)[k], axis=1).max() * np.abs(p.clean(p.dout)[q]).max() * \
                np.sqrt(d)
            err = np.linalg.norm(dq[q] - ref[0][q])
            assert err <= 2.0 ** -7 * np.linalg.norm(ref[0][q]) + \
                2.0 ** -16 * size * np.sqrt(nq * heads), nk


def test_bounds_do_not_change_bits():
    """The same sequences with bounds that hold them and with larger ones."""
    lens, sq = [5, 100, 128, 17], 50
    off, q_off = offsets(lens), offsets([sq] * 4)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    p = Problem(4, 4 * sq, off[-1], 4, 2, 64, q_offsets=q_off, kv_offsets=off, max_q=sq,
                max_kv=128).check_forward()
    rows = dict(n=4, q_offsets=i32(q_off), kv_offsets=i32(off))
    first = backward(p, (0, 4 * sq), (0, off[-1]), max_q=sq, max_kv=128, **rows)
    for bounds in (dict(max_q=sq, max_kv=129), dict(max_q=4 * sq), {}):
        again = backward(p, (0, 4 * sq), (0, off[-1]), **bounds, **rows)
        assert all(torch.equal(x, y) for x, y in zip(first, again)), bounds


# a cluster shares the queries of a key block (few key blocks, many queries), of which
# some hold all keys of their sequence and some do not
SHARED = [(2, 1500, 300, 2, 1, 128, [300, 9]), (3, 1100, 200, 4, 1, 64, [128, 200, 2]),
          (1, 4000, 131, 2, 2, 64, [3]), (4, 700, 260, 3, 1, 128, [1, 129, 0, 128])]


def shared(n, sq, sk, heads, kv_heads, d, lens):
    return Problem(n, n * sq, n * sk, heads, kv_heads, d, kv_lens=lens,
                   q_lens=[sq - 7 * i for i in range(n)])


@pytest.mark.parametrize("case", SHARED)
def test_shares_of_queries(case):
    p = shared(*case).check()
    first = p.dq_all.clone(), p.dkv_all.clone()
    for _ in range(3):
        p.backward()
        assert torch.equal(p.dq_all, first[0]) and torch.equal(p.dkv_all, first[1])


def results():
    """Digests of the gradients (a call's status is checked) in this build."""
    out = []
    for p in [shared(*c) for c in SHARED] + list(problems(128, 6, 2, 33)):
        p.forward()
        p.backward()
        out.append(digest(p.o_all, p.lse, p.dq_all, p.dkv_all))
    return out


def test_debug_build_is_clean_and_matches_release():
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "from megatron_transformer_layer_gb300 import _lib as L\n"
            "assert L.LIB_PATH.endswith('_debug.so')\n"
            "from test_gpu_cross_attention_short import results\n"
            "for r in results(): print(r)\n") % (os.path.dirname(TESTS), TESTS)
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600,
                         env=dict(os.environ, MC_LAYER_DEBUG="1"))
    assert out.returncode == 0, out.stderr[-2000:]
    assert out.stdout.split() == results()
