"""Attention to keys of another length and the norms of queries and keys in the debug
build: its index checks pass at ragged shapes, in every instance of the kernels, and
the results are the release build's to the bit."""
import os
import subprocess
import sys

import pytest
import torch

import test_gpu_cross_attention as C
import test_gpu_qk_norm as N
from gpu_util import status
from test_gpu_attention_opt_debug import TESTS, digest
from megatron_transformer_layer_gb300 import _lib as L

pytestmark = pytest.mark.gpu

CROSS = [  # n, query rows, key rows, heads, key heads, head_dim, more
    (3, 3, 4500, 4, 1, 64, {}),                        # shares of the keys
    (2, 2, 5000, 2, 2, 128, {}),
    (1, 1500, 130, 2, 1, 128, {}),                     # shares of the queries
    (1, 1300, 90, 4, 1, 64, {}),
    (3, 400, 900, 6, 2, 64, dict(q_offsets=[0, 129, 140, 400], kv_offsets=[0, 1, 600, 880],
                                 q_lens=[129, 0, 250], kv_lens=[1, 500, 280], wide=128)),
    (3, 400, 900, 6, 2, 128, dict(q_offsets=[0, 129, 140, 400], kv_offsets=[0, 1, 600, 880],
                                  kv_lens=[1, 500, 0], max_q=300, max_kv=600)),
    (70, 70 * 130, 70 * 140, 5, 5, 64, dict(kv_lens=[3 * k % 141 for k in range(70)])),
    (40, 40 * 30, 40 * 140, 10, 2, 128, {}),
]
NORM = [  # tokens, heads of queries and of keys, head_dim, more
    (9, 3, 1, 64, dict(rot=64)), (1, 2, 2, 128, {}), (700, 16, 4, 128, dict(rot=64, centred=True, adjacent=True)),
    (333, 2, 0, 96, dict(rot=30, dtype=torch.float32, extra=1)),
    (50, 0, 5, 7, dict(centred=True, gains=False)), (4100, 8, 8, 64, dict(rot=64, dtype=torch.float32))]


def cross(case):
    p = C.Problem(*case[:6], **case[6])
    st = status()
    assert L.mc_attention_forward_cross(p.q, p.k, p.v, p.o, p.lse, p.cross, st) == 0
    p.backward()
    return int(st[0]), digest(p.o_all, p.lse, p.dq_all, p.dkv_all)


def norm(case):
    p = N.Problem(*case[:4], **case[4])
    st, w = status(), p.H * p.d
    out = torch.zeros(p.tokens, w, dtype=p.dtype, device=p.x.device)
    assert L.mc_qk_norm_forward(p.x, out, *p.heads(), p.ld, w, p.norm, p.positions, p.inv_freq, p.spec,
                                st) == 0
    g = [torch.zeros(p.d, device=p.x.device) for _ in range(4)]
    din = p.backward(L.make_qk_norm_grads(*g))
    return int(st[0]), digest(out, din, *g)


def results():
    return [f(c) for f, cases in ((cross, CROSS), (norm, NORM)) for c in cases]


def test_debug_build_is_clean_and_matches_release():
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "from megatron_transformer_layer_gb300 import _lib as L\n"
            "assert L.LIB_PATH.endswith('_debug.so')\n"
            "from test_gpu_cross_attention_debug import results\n"
            "for r in results(): print(*r)\n") % (os.path.dirname(TESTS), TESTS)
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600,
                         env=dict(os.environ, MC_LAYER_DEBUG="1"))
    assert out.returncode == 0, out.stderr[-2000:]
    debug = [line.split() for line in out.stdout.strip().splitlines()]
    assert len(debug) == len(CROSS + NORM)
    for case, (code, sha), (rcode, rsha) in zip(CROSS + NORM, debug, results()):
        assert int(code) == rcode == 0, case
        assert sha == rsha, case
