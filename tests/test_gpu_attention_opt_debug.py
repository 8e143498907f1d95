"""Positions, masks and attention over them in the debug build: its index checks
pass at ragged shapes, in every instance of the kernels, and the results are the
release build's to the bit."""
import hashlib
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from megatron_transformer_layer_gb300 import _lib as L

from gpu_util import DEV, status
from test_gpu_attention_opt import Problem, gen, i32

pytestmark = pytest.mark.gpu

TESTS = os.path.dirname(os.path.abspath(__file__))
ROTARY = [  # tokens, heads, head_dim, rot_dim, adjacent pairs, type, in place
    (7, 3, 128, 64, False, torch.bfloat16, False), (130, 5, 128, 64, True, torch.bfloat16, False),
    (9, 1, 6, 2, False, torch.float32, True), (4, 2, 96, 60, True, torch.bfloat16, True),
    (600, 64, 128, 128, False, torch.bfloat16, True), (11, 3, 80, 36, False, torch.bfloat16, False)]
MASKS = [(1, 1, 1), (2, 300, 5), (9, 4100, 60), (4200, 7, 4000)]  # b, s, documents
ATTENTION = [(kind, b, s, H, d, cap, bias)
             for cap, bias in ((0.0, False), (4.0, False), (0.0, True), (4.0, True))
             for kind, b, s, H, d in (("documents", 2, 333, 2, 128), ("any", 1, 450, 3, 64),
                                      ("nothing", 1, 129, 2, 64))] + \
    [("window", 6, 1200, 12, 64, 0.0, False), ("prefix", 37, 3, 2, 128, 0.0, True)]


def digest(*tensors):
    h = hashlib.sha256()
    for t in tensors:
        h.update(t.contiguous().view(torch.uint8).cpu().numpy().tobytes())
    return h.hexdigest()


def rotary(case):
    tokens, heads, d, rot, adjacent, dtype, in_place = case
    g = gen(tokens)
    x = torch.randn(tokens, heads * d + 3, generator=g).to(dtype).to(DEV)
    out = x if in_place else torch.full_like(x, 7.0)
    pos = torch.randint(-9, 5000, (1, tokens), generator=g, dtype=torch.int32).to(DEV)
    freq, st = torch.rand(rot // 2, generator=g).to(DEV), status()
    for call in (L.mc_rotary_forward, L.mc_rotary_backward):
        assert call(x, out, tokens, heads, d, x.shape[1], x.shape[1], pos, freq,
                    L.make_rotary_spec(rot, None, adjacent), st) == 0
    return int(st[0]), digest(out)


def mask(case):
    b, s, docs = case
    cuts = np.sort(np.random.default_rng(s).integers(0, b * s + 1, docs + 1))
    lo, hi = (torch.full((b, s), -7, dtype=torch.int32, device=DEV) for _ in range(2))
    tab = torch.full((2, L.mc_attention_mask_table_ints(b, s)), -7, dtype=torch.int32, device=DEV)
    st = status()
    assert L.mc_attention_mask_documents(i32(cuts), docs, None, 1, 90, b, s, lo, hi, tab[0], st) == 0
    assert L.mc_attention_mask_intervals(b, s, lo, hi, tab[1], st) == 0
    assert torch.equal(tab[0], tab[1])
    return int(st[0]), digest(lo, hi, tab)


def attention(case):
    p, st = Problem(*case), status()
    assert L.mc_attention_forward_opt(p.qkv, p.o, p.lse, p.b, p.s, p.H, p.d, p.opt, st) == 0
    out = [p.o, p.lse]
    n = L.mc_attention_backward_opt_ws_bytes(p.b, p.s, p.H, p.d, p.opt)
    for ws in (None, torch.empty(n, dtype=torch.uint8, device=DEV)):
        out.append(torch.full_like(p.qkv, 3.0))
        assert L.mc_attention_backward_opt(p.qkv, p.o, p.lse, p.dout, out[-1], p.delta, p.b, p.s,
                                           p.H, p.d, p.opt, ws, n if ws is not None else 0, st) == 0
    return int(st[0]), digest(*out)


def results():
    return [f(c) for f, cases in ((rotary, ROTARY), (mask, MASKS), (attention, ATTENTION))
            for c in cases]


def test_debug_build_is_clean_and_matches_release():
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "from megatron_transformer_layer_gb300 import _lib as L\n"
            "assert L.LIB_PATH.endswith('_debug.so')\n"
            "from test_gpu_attention_opt_debug import results\n"
            "for r in results(): print(*r)\n") % (os.path.dirname(TESTS), TESTS)
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600,
                         env=dict(os.environ, MC_LAYER_DEBUG="1"))
    assert out.returncode == 0, out.stderr[-2000:]
    debug = [line.split() for line in out.stdout.strip().splitlines()]
    cases = ROTARY + MASKS + ATTENTION
    assert len(debug) == len(cases)
    for case, (code, sha), (rcode, rsha) in zip(cases, debug, results()):
        assert int(code) == rcode == 0, case
        assert sha == rsha, case
