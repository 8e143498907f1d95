"""Attention to keys and values of another length on the GPU, against the float64
oracle.  Tolerances are the oracle's: counted per element from the roundings of a
bf16 pipeline (half a step, 2^-8, where P, dz and the results are stored) and
2^-16 for 32-bit arithmetic, before the first run."""
import numpy as np
import pytest
import torch

import oracle.cross_attention as O
from megatron_transformer_layer_gb300 import _lib as L

from gpu_util import DEV, check_status, status, to_f64

pytestmark = pytest.mark.gpu

KEEP = 3.0  # what is in the buffers before a call


def i32(x):
    return None if x is None else torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Problem:
    """One problem on the GPU, and its oracle.  `hole`: what lies in the rows that
    nothing may read (padding, between and behind the sequences)."""

    def __init__(self, n, q_rows, k_rows, heads, kv_heads, d, q_offsets=None, q_lens=None,
                 kv_offsets=None, kv_lens=None, scale=0.0, max_q=0, max_kv=0, wide=0, qstd=1.5,
                 hole=float("nan"), seed=0):
        g = torch.Generator().manual_seed(seed + q_rows + k_rows)
        self.n, self.heads, self.kv_heads, self.d = n, heads, kv_heads, d
        self.q_rows, self.k_rows = q_rows, k_rows
        self.q_seq = O.sequence_rows(n, q_rows, q_offsets, q_lens)
        self.k_seq = O.sequence_rows(n, k_rows, kv_offsets, kv_lens)
        a, akv = heads * d, kv_heads * d
        self.a, self.akv, self.wide = a, akv, wide

        def make(rows, width, std, seq):
            x = torch.randn(rows, width, generator=g) * std
            live = torch.zeros(rows, dtype=torch.bool)
            for first, _, real in seq:
                live[first: first + real] = True
            x[~live] = hole
            return x.bfloat16().to(DEV)

        # rows of Q, of K | V and of O may be wider than their heads
        self.q_all = make(q_rows, a + wide, qstd, self.q_seq)
        self.kv_all = make(k_rows, 2 * akv + wide, 1.0, self.k_seq)
        self.do_all = make(q_rows, a + 2 * wide, 1.0, self.q_seq)
        self.q, self.dout = self.q_all[:, :a], self.do_all[:, :a]
        self.k, self.v = self.kv_all[:, :akv], self.kv_all[:, akv: 2 * akv]
        self.o_all = torch.full((q_rows, a + 2 * wide), KEEP, dtype=torch.bfloat16, device=DEV)
        self.o = self.o_all[:, :a]
        self.lse = torch.full((heads, q_rows), KEEP, device=DEV)
        self.cross = L.make_cross_attention(
            n, q_rows, k_rows, heads, kv_heads, d, ld_q=a + wide, ld_kv=2 * akv + wide,
            ld_o=a + 2 * wide, q_offsets=i32(q_offsets), q_lens=i32(q_lens),
            kv_offsets=i32(kv_offsets), kv_lens=i32(kv_lens), max_q=max_q, max_kv=max_kv,
            scale=scale)
        self.scale = scale or O.default_scale(d)

    def clean(self, x):
        return np.nan_to_num(to_f64(x), nan=0.0, posinf=0.0, neginf=0.0)

    def forward(self, stream=None):
        st = status()
        assert L.mc_attention_forward_cross(self.q, self.k, self.v, self.o, self.lse, self.cross, st,
                                            stream) == 0
        check_status(st)

    def check_forward(self):
        self.forward()
        o, lse, tol, ltol, owned = O.forward(self.clean(self.q), self.clean(self.k),
                                             self.clean(self.v), self.q_seq, self.k_seq, self.heads,
                                             self.kv_heads, self.d, self.scale)
        got, glse = to_f64(self.o_all), to_f64(self.lse)
        assert (got[~owned] == KEEP).all() and (glse[:, ~owned] == KEEP).all()
        assert (got[:, self.a:] == KEEP).all()
        off = (np.abs(got[:, : self.a] - o) / tol)[owned]
        assert np.isfinite(got).all()
        if off.size:
            assert off.max() <= 1, f"O: {off.max():.3g} of the tolerance"
        seen = np.isfinite(lse) & owned
        blank = ~np.isfinite(lse) & owned
        assert (glse[blank] == -np.inf).all()
        if seen.any():
            off = np.abs(glse[seen] - lse[seen]) / ltol[seen]
            assert off.max() <= 1, f"lse: {off.max():.3g} of the tolerance"
        return self

    def backward(self):
        """dq, dk, dv [rows, ...] of NaN-free buffers whose other places stay as they were."""
        c = self.cross
        self.dq_all = torch.full_like(self.q_all, KEEP)
        self.dkv_all = torch.full_like(self.kv_all, KEEP)
        delta = torch.empty(self.heads, self.q_rows, device=DEV)
        n = L.mc_attention_backward_cross_ws_bytes(c)
        ws = torch.full((n + 256,), 0xff, dtype=torch.uint8, device=DEV)  # NaN
        st = status()
        dk, dv = self.dkv_all[:, : self.akv], self.dkv_all[:, self.akv: 2 * self.akv]
        assert L.mc_attention_backward_cross(self.q, self.k, self.v, self.o, self.lse, self.dout,
                                             self.dq_all[:, : self.a], dk, dv, delta, c, ws, n,
                                             st) == 0
        check_status(st)
        assert (ws[n:] == 0xff).all()
        return self.dq_all[:, : self.a], dk, dv

    def check_backward(self):
        ref, tol, t32 = O.backward(*map(self.clean, (self.q, self.k, self.v, self.dout)),
                                   self.q_seq, self.k_seq, self.heads, self.kv_heads, self.d,
                                   self.scale)
        got = [to_f64(x) for x in self.backward()]
        for name, g, r, t, e, seq in zip(("dQ", "dK", "dV"), got, ref, tol, t32,
                                         (self.q_seq, self.k_seq, self.k_seq)):
            owned = np.zeros(len(g), dtype=bool)
            for first, slot, real in seq:
                owned[first: first + slot] = True
                assert (g[first + real: first + slot] == 0).all(), name
            assert (g[~owned] == KEEP).all(), name
            if owned.any():
                off = (np.abs(g - r) / t)[owned]
                assert off.max() <= 1, f"{name}: {off.max():.3g} of the tolerance"
                # roundings of either sign: the 2-norm within two of them, and the
                # 32-bit part (see the other attention's test)
                assert np.linalg.norm((g - r)[owned]) <= \
                    2 * O.HALF_BF16 * np.linalg.norm(r) + np.linalg.norm(e), name
        assert (to_f64(self.dq_all)[:, self.a:] == KEEP).all()
        assert (to_f64(self.dkv_all)[:, 2 * self.akv:] == KEEP).all()
        return self

    def check(self):
        return self.check_forward().check_backward()


# ------------------------------------------------------------------ forward and backward
@pytest.mark.parametrize("sq,sk", [(1, 1), (1, 127), (2, 128), (127, 129), (128, 255), (129, 256),
                                   (200, 257), (64, 400), (300, 1), (1, 3000), (260, 700)])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths(sq, sk, d):
    Problem(1, sq, sk, 2, 2, d).check()


@pytest.mark.parametrize("heads,kv_heads", [(3, 3), (6, 2), (5, 1), (8, 1), (12, 4), (7, 1), (48, 1),
                                            (100, 1), (128, 1), (16, 8)])
@pytest.mark.parametrize("sq,sk", [(1, 300), (5, 130), (70, 390)])
def test_grouped_heads(heads, kv_heads, sq, sk):
    Problem(2, 2 * sq, 2 * sk, heads, kv_heads, 64, kv_lens=[sk, sk // 3]).check()


def test_grouped_heads_of_128():
    Problem(3, 3 * 33, 3 * 300, 8, 2, 128, kv_lens=[300, 1, 129], wide=128).check()


@pytest.mark.parametrize("d", [64, 128])
def test_padded(d):
    """Padded keys and queries hold NaN; a sequence has no keys, another no queries."""
    Problem(5, 5 * 150, 5 * 300, 4, 2, d, q_lens=[150, 1, 0, 77, 128],
            kv_lens=[300, 0, 256, 1, 299], wide=128).check()
    Problem(5, 5 * 150, 5 * 300, 3, 3, d, q_lens=[150, 1, 0, 77, 128],
            kv_lens=[300, 0, 256, 1, 299], wide=8).check()


@pytest.mark.parametrize("d", [64, 128])
def test_packed(d):
    Problem(6, 700, 900, 4, 4, d, q_offsets=[3, 3, 130, 131, 400, 640, 690],
            kv_offsets=[10, 300, 300, 301, 557, 700, 890]).check()
    Problem(6, 700, 900, 4, 2, d, q_offsets=[3, 3, 130, 131, 400, 640, 690], max_q=300, max_kv=290,
            kv_offsets=[10, 300, 300, 301, 557, 700, 890]).check()


def test_packed_with_padding_inside():
    Problem(3, 500, 600, 2, 1, 128, q_offsets=[0, 200, 260, 480], q_lens=[180, 60, 0],
            kv_offsets=[0, 100, 400, 590], kv_lens=[99, 300, 20]).check()


def test_infinities_in_the_padding():
    Problem(4, 4 * 20, 4 * 200, 2, 2, 64, kv_lens=[200, 100, 0, 129], q_lens=[20, 3, 20, 1],
            hole=float("inf")).check()


def test_offsets_outside_the_rows_are_cut():
    Problem(3, 100, 100, 2, 2, 64, q_offsets=[-5, 40, 90, 1000], q_lens=[7, -3, 50],
            kv_offsets=[-2 ** 31, 10, 90, 2 ** 31 - 1], kv_lens=[2 ** 31 - 1] * 3,
            hole=0.0).check()


def test_a_sequence_longer_than_stated_is_reported():
    p = Problem(2, 400, 300, 2, 2, 64, q_offsets=[0, 250, 400], kv_offsets=[0, 100, 300], max_q=200,
                max_kv=200)
    st = status()
    assert L.mc_attention_forward_cross(p.q, p.k, p.v, p.o, p.lse, p.cross, st) == 0
    torch.cuda.synchronize()
    assert int(st[0]) == L.MC_ERR_DEVICE_BOUNDS
    Problem(1, 40, 40, 2, 2, 64).check()  # the next call is as ever


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sq,sk,heads,kv_heads", [(300, 1, 2, 2), (1, 1, 12, 12), (300, 2, 4, 2),
                                                  (40, 3, 8, 8), (1500, 9, 2, 1), (130, 128, 3, 3)])
def test_gradients_with_few_keys(d, sq, sk, heads, kv_heads):
    """Where a sequence has few keys dP - delta cancels: what is left has to be as
    exact as elsewhere, roundings to bf16 of dz and of dQ (each at most 2^-8 of the
    value, so that together they stay below 2^-7 of the 2-norm), beside 2^-16 of the
    terms' size (delta, P and lse in 32 bits).  With one key dQ is 0."""
    n = 3
    p = Problem(n, n * sq, n * sk, heads, kv_heads, d, q_lens=[sq, max(1, sq - 7), sq],
                kv_lens=[sk, max(1, sk - 1), sk]).check_forward()
    dq = to_f64(p.check_backward().dq_all)[:, : p.a]
    ref, _, _ = O.backward(*map(p.clean, (p.q, p.k, p.v, p.dout)), p.q_seq, p.k_seq, heads, kv_heads,
                           d, p.scale)
    size = p.scale * np.linalg.norm(p.clean(p.k), axis=1).max() * \
        np.linalg.norm(p.clean(p.v), axis=1).max() * np.abs(p.clean(p.dout)).max() * np.sqrt(d)
    err = np.linalg.norm((dq - ref[0])[[i for f, _, r in p.q_seq for i in range(f, f + r)]])
    rows = np.sqrt(sum(r for _, _, r in p.q_seq) * heads)
    assert err <= 2.0 ** -7 * np.linalg.norm(ref[0]) + 2.0 ** -16 * size * rows
    if sk == 1:
        assert (dq == 0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_one_key_beside_many(d):
    """A sequence's only key has the weight 1: no gradient of its queries, in a call
    whose other sequences have many keys too."""
    p = Problem(3, 3 * 140, 3 * 300, 4, 2, d, kv_lens=[300, 1, 129]).check()
    dq = to_f64(p.dq_all)[140:280, : p.a]
    assert (dq == 0).all()
    assert (to_f64(p.dkv_all)[300, : p.akv] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("wide", [8, 24])
def test_rows_of_other_widths(d, wide):
    """Strides that are multiples of 8 elements only."""
    Problem(2, 300, 400, 3, 3, d, q_lens=[150, 3], kv_lens=[130, 200], wide=wide).check()


@pytest.mark.parametrize("scale", [1.0, 0.01, 2.0 ** -16])
def test_scale(scale):
    Problem(1, 130, 300, 2, 2, 64, scale=scale, qstd=0.5).check()


def test_growing_scores():
    """Maxima that grow from block to block, so that O is rescaled."""
    p = Problem(1, 140, 2000, 2, 2, 128, qstd=1.0)
    p.kv_all[:, : p.akv] *= torch.linspace(0.1, 8.0, 2000, device=DEV).bfloat16()[:, None]
    p.check()


def test_many_items():
    """More items than SMs hold at once: blocks taken over by running CTAs."""
    Problem(40, 40 * 130, 40 * 70, 9, 9, 64, kv_lens=[1 + (i * 37) % 70 for i in range(40)],
            q_lens=[130 - (i * 11) % 130 for i in range(40)]).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("more", [0, 128, 300, 1000])
@pytest.mark.parametrize("sq,heads,kv_heads", [(1, 8, 8), (3, 16, 8)])
def test_ends_of_sequences(d, more, sq, heads, kv_heads):
    """Last blocks of every kind, where items fill the SMs."""
    ends = [1, 15, 16, 17, 32, 33, 64, 96, 97, 127, 128, 0]
    lens = [n + more * (k % 3 != 1) for k, n in enumerate(ends)]
    rows = 128 + more
    Problem(len(ends), len(ends) * sq, len(ends) * rows, heads, kv_heads, d, kv_lens=lens).check()


@pytest.mark.parametrize("n,sk,heads,kv_heads,d", [(1, 8191, 8, 1, 128), (2, 4097, 4, 4, 64),
                                                   (3, 2049, 6, 2, 128), (9, 600, 8, 8, 64)])
def test_one_token_long_states(n, sk, heads, kv_heads, d):
    """Few rows: the keys of an item are shared out."""
    Problem(n, n, n * sk, heads, kv_heads, d,
            kv_lens=[max(0, sk - 700 * i) for i in range(n)]).check()


@pytest.mark.parametrize("n,sq,sk,heads,kv_heads,d", [(1, 1500, 130, 2, 1, 128), (2, 700, 100, 4, 1, 64),
                                                      (1, 4000, 60, 2, 2, 64), (3, 900, 257, 3, 1, 128)])
def test_many_queries_few_keys(n, sq, sk, heads, kv_heads, d):
    """Few key blocks: the queries of an item are shared out in the backward pass."""
    Problem(n, n * sq, n * sk, heads, kv_heads, d, q_lens=[max(1, sq - 650 * i) for i in range(n)],
            kv_lens=[sk - 29 * i for i in range(n)], wide=64 * (d // 64)).check()


def test_same_bits_again():
    for p in (Problem(2, 2 * 30, 2 * 3000, 4, 2, 128, kv_lens=[3000, 1234]),
              Problem(1, 2000, 200, 4, 2, 64),
              Problem(20, 20 * 300, 20 * 260, 6, 6, 64, kv_lens=[13 * i for i in range(20)])):
        p.forward()
        o, lse = p.o.clone(), p.lse.clone()
        first = [x.clone() for x in p.backward()]
        for _ in range(3):
            p.forward()
            assert torch.equal(p.o, o) and torch.equal(p.lse, lse)
            assert all(torch.equal(x, y) for x, y in zip(p.backward(), first))


def test_heads_in_groups():
    """Packed sequences whose longest is not known: the tiles of one key head fill
    the workspace, the heads take turns."""
    n, rows = 150, 2900
    cuts = [rows * i // n for i in range(n + 1)]
    p = Problem(n, rows, rows + 40, 6, 3, 64, q_offsets=cuts, kv_offsets=[c + 10 for c in cuts])
    per_head = n * ((rows + 63) // 64) * ((rows + 40 + 127) // 128) * 32768
    assert L.mc_attention_backward_cross_ws_bytes(p.cross) == per_head > 2 ** 30
    p.check()


def test_nan_in_a_real_key_stays_in_its_sequence():
    p = Problem(3, 3 * 40, 3 * 300, 2, 2, 64, hole=0.0)
    p.forward()
    o = p.o.clone()
    p.v[350, :] = float("nan")
    p.forward()
    assert torch.isnan(p.o[40:80].float()).all()
    assert torch.equal(p.o[:40], o[:40]) and torch.equal(p.o[80:], o[80:])
