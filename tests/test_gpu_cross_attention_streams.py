"""Attention to keys of another length and the norms of queries and keys as programs
run them: without a stream argument, captured and replayed (lengths changed in
between, too), on two streams at once, in two graphs that share a workspace, far into
a long cache.  Every call is compared with the same call alone, to the bit."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_gb300 import _lib as L

from gpu_util import DEV, check_status, status
from test_gpu_attention_opt import bf16, gen, i32
from test_gpu_attention_opt_streams import replayed, same

pytestmark = pytest.mark.gpu


class Attention:
    """A problem's tensors and calls; the workspace may be another one's."""

    def __init__(self, n, sq, sk, heads, kv_heads, d, lens=None, seed=0, ws=None, packed=False):
        a, akv = heads * d, kv_heads * d
        self.st = status()
        self.q, self.dout = bf16(gen(seed + 1), n * sq, a), bf16(gen(seed + 2), n * sq, a)
        self.kv = bf16(gen(seed + 3), n * sk, 2 * akv)
        self.k, self.v = self.kv[:, :akv], self.kv[:, akv:]
        self.lens = None if lens is None else i32(lens)
        off = i32(np.arange(n + 1) * sk) if packed else None
        self.c = L.make_cross_attention(n, n * sq, n * sk, heads, kv_heads, d, ld_kv=2 * akv,
                                        kv_lens=self.lens, kv_offsets=off, max_kv=sk if packed else 0)
        self.o, self.dq = torch.zeros_like(self.q), torch.zeros_like(self.q)
        self.dkv = torch.zeros_like(self.kv)
        self.lse, self.delta = (torch.zeros(heads, n * sq, device=DEV) for _ in range(2))
        self.n = L.mc_attention_backward_cross_ws_bytes(self.c)
        self.ws = torch.empty(self.n, dtype=torch.uint8, device=DEV) if ws is None else ws
        assert self.ws.numel() >= self.n
        self.akv = akv

    def forward(self, stream=None):
        return L.mc_attention_forward_cross(self.q, self.k, self.v, self.o, self.lse, self.c, self.st,
                                            stream)

    def backward(self, stream=None):
        return L.mc_attention_backward_cross(self.q, self.k, self.v, self.o, self.lse, self.dout,
                                             self.dq, self.dkv[:, : self.akv],
                                             self.dkv[:, self.akv:], self.delta, self.c, self.ws,
                                             self.n, self.st, stream)

    def step(self, stream=None):
        return [self.forward(stream), self.backward(stream)]

    def outputs(self):
        return [self.o, self.lse, self.dq, self.dkv]

    def alone(self):
        """The outputs of one step, which are then cleared."""
        assert self.step() == [0, 0]
        torch.cuda.synchronize()
        want = [x.clone() for x in self.outputs()]
        self.clear()
        return want

    def clear(self):
        for x in self.outputs():
            x.zero_()
        torch.cuda.synchronize()


class Norm:
    def __init__(self, tokens=700, q_heads=6, k_heads=2, d=128, seed=0):
        H = q_heads + k_heads
        self.st = status()
        self.x, self.dout = bf16(gen(seed + 1), tokens, H * d), bf16(gen(seed + 2), tokens, H * d)
        self.out, self.din = torch.zeros_like(self.x), torch.zeros_like(self.x)
        self.norm = L.make_qk_norm(bf16(gen(seed + 3), d), bf16(gen(seed + 4), d))
        self.g = [torch.zeros(d, device=DEV) for _ in range(2)]
        self.grads = L.make_qk_norm_grads(q_gain=self.g[0], k_gain=self.g[1])
        self.scratch = torch.empty(L.mc_qk_norm_scratch_floats(tokens, q_heads, k_heads, d), device=DEV)
        self.heads, self.ld = (tokens, q_heads, k_heads, d), H * d
        self.turn = (i32(np.arange(tokens)[None]), torch.rand(d // 2, generator=gen(seed + 5)).to(DEV),
                     L.make_rotary_spec(d))

    def step(self, stream=None):
        ld = self.ld
        return [L.mc_qk_norm_forward(self.x, self.out, *self.heads, ld, ld, self.norm, *self.turn,
                                     self.st, stream),
                L.mc_qk_norm_backward(self.x, self.dout, self.din, *self.heads, ld, ld, ld, self.norm,
                                      *self.turn, self.grads, 0, self.scratch, self.st, stream)]

    def outputs(self):
        return [self.out, self.din, *self.g]

    alone, clear = Attention.alone, Attention.clear


PROBLEMS = [  # one token with shares of the keys, many items, and shares of the queries
    lambda **kw: Attention(3, 1, 2000, 4, 1, 64, **kw),
    lambda **kw: Attention(9, 130, 300, 6, 3, 128, [300, 7, 0, 299, 128, 129, 1, 256, 257], **kw),
    lambda **kw: Attention(1, 1500, 130, 2, 1, 128, **kw),
    lambda **kw: Attention(2, 70, 90, 16, 16, 64, **kw)]


@pytest.mark.parametrize("make", PROBLEMS + [Norm])
def test_calls_without_a_stream(make):
    p = make()
    assert same(replayed(p.step, p.outputs()))
    check_status(p.st)


@pytest.mark.parametrize("first,second", [(0, 1), (1, 1), (1, 2), (0, 0), (3, 1)])
def test_two_streams_at_once(first, second):
    a, b = PROBLEMS[first](), PROBLEMS[second](seed=50)
    n, m = Norm(), Norm(3000, 16, 16, 64, seed=70)
    sides = [torch.cuda.Stream() for _ in range(2)]
    want = [p.alone() for p in (a, n, b, m)]
    for _ in range(10):
        for side, pair in zip(sides, ((a, n), (b, m))):
            for p in pair:
                assert p.step(side) == [0, 0]
    torch.cuda.synchronize()
    for p, w in zip((a, n, b, m), want):
        assert all(torch.equal(x, y) for x, y in zip(p.outputs(), w))
        check_status(p.st)


def capture(call):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        assert call() == [0, 0]
    torch.cuda.synchronize()
    return graph


def test_two_graphs_share_a_workspace():
    """Replayed one after the other on a stream, as a program of two layers would."""
    big = PROBLEMS[1]()
    small = PROBLEMS[2](seed=50, ws=big.ws)
    n = Norm()
    m = Norm(seed=70)
    m.scratch = n.scratch
    parts = (big, small, n, m)
    want = [p.alone() for p in parts]
    graphs = [capture(p.step) for p in parts]
    for order in ((0, 1, 2, 3), (1, 0, 3, 2), (0, 0, 1, 1)):
        for p in parts:
            p.clear()
        big.ws.fill_(0xff)
        n.scratch.fill_(float("nan"))
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize()
        for k in set(order):
            assert all(torch.equal(x, y) for x, y in zip(parts[k].outputs(), want[k]))


def test_lengths_change_between_replays():
    """Lengths are read by the kernels: a captured decoding step follows them."""
    lens = [[1, 500, 64], [2, 501, 65], [0, 700, 1], [700, 700, 700]]
    for sq, packed in ((1, False), (40, True)):
        p = Attention(3, sq, 700, 4, 2, 64, lens[0], packed=packed)
        want = []
        for now in lens:
            p.lens.copy_(i32(now))
            want.append(p.alone())
        graph = capture(p.step)
        for now, w in zip(lens, want):
            p.lens.copy_(i32(now))
            p.clear()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(p.outputs(), w))
        check_status(p.st)


def test_the_same_tensor_as_keys_and_values():
    p = Attention(2, 50, 170, 4, 2, 128)
    p.v = p.k
    twin = Attention(2, 50, 170, 4, 2, 128)
    twin.kv[:, twin.akv:] = twin.kv[:, : twin.akv]
    for x, y in zip(p.alone(), twin.alone()):
        assert torch.equal(x, y)


@pytest.mark.parametrize("sq,sk", [(1, 300), (100, 300)])
def test_rows_past_32_bits(sq, sk):
    """Sequences that lie behind 2^31 elements of their tensors give the bits of the
    same ones in tensors of their own."""
    heads, kv_heads, d, ld, rows = 4, 2, 64, 16384, 140000
    near = Attention(1, sq, sk, heads, kv_heads, d)
    want = near.alone()
    a, akv = near.q.shape[1], near.akv
    # (Q, dO, K and V in columns of one tensor; O, dQ, dK and dV of another)
    ins = torch.zeros(rows, ld, dtype=torch.bfloat16, device=DEV)
    outs = torch.full((rows, ld), 3.0, dtype=torch.bfloat16, device=DEV)
    q0, k0 = rows - sq, rows - sk
    assert k0 * ld > 2 ** 31
    cut = lambda t, at, w: t[:, at: at + w]  # noqa: E731
    q, dout, k, v = cut(ins, 0, a), cut(ins, a, a), cut(ins, 2 * a, akv), cut(ins, 2 * a + akv, akv)
    o, dq, dk, dv = cut(outs, 0, a), cut(outs, a, a), cut(outs, 2 * a, akv), \
        cut(outs, 2 * a + akv, akv)
    q[q0:], dout[q0:], k[k0:], v[k0:] = near.q, near.dout, near.k, near.v
    c = L.make_cross_attention(1, rows, rows, heads, kv_heads, d, ld_q=ld, ld_kv=ld, ld_o=ld,
                               q_offsets=i32([q0, rows]), kv_offsets=i32([k0, rows]), max_q=sq,
                               max_kv=sk)
    lse, delta = (torch.zeros(heads, rows, device=DEV) for _ in range(2))
    st, n = status(), L.mc_attention_backward_cross_ws_bytes(c)
    assert n == near.n
    assert L.mc_attention_forward_cross(q, k, v, o, lse, c, st) == 0
    assert L.mc_attention_backward_cross(q, k, v, o, lse, dout, dq, dk, dv, delta, c, near.ws, n,
                                         st) == 0
    check_status(st)
    got = [o[q0:], lse[:, q0:], dq[q0:], torch.cat([dk[k0:], dv[k0:]], 1)]
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert (outs[: k0] == 3.0).all() and (outs[:, 2 * a + 2 * akv:] == 3.0).all()


def test_a_backward_pass_longer_than_stated_is_reported():
    p = Attention(1, 200, 400, 2, 2, 64)
    assert p.forward() == 0
    for kw in (dict(kv_offsets=i32([0, 400]), max_kv=128), dict(q_offsets=i32([0, 200]), max_q=100)):
        st = status()
        c = L.make_cross_attention(1, 200, 400, 2, 2, 64, ld_kv=256, **kw)
        n = L.mc_attention_backward_cross_ws_bytes(c)
        ws = torch.zeros(n + 4096, dtype=torch.uint8, device=DEV)
        assert L.mc_attention_backward_cross(p.q, p.k, p.v, p.o, p.lse, p.dout, p.dq, p.dkv[:, :128],
                                             p.dkv[:, 128:], p.delta, c, ws, n, st) == 0
        torch.cuda.synchronize()
        assert int(st[0]) == L.MC_ERR_DEVICE_BOUNDS
        assert not ws[n:].any()
