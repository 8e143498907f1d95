"""Rotary positions, interval masks and attention over them on the GPU, each
against the float64 oracle.  Tolerances are the oracle's: counted per element
from the roundings of a bf16 pipeline (half a step, 2^-8, where P, dz and the
results are stored) and 2^-16 for 32-bit arithmetic, before the first run."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle.attention_opt as O
from megatron_transformer_layer_gb300 import _lib as L

from gpu_util import DEV, check_status, status, to_f64

pytestmark = pytest.mark.gpu


def bf16(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).bfloat16().to(DEV)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ rotary
@pytest.mark.parametrize("tokens,heads,d,rot,sections,adjacent,dealt,dtype,extra", [
    (1, 24, 64, 64, None, False, False, torch.bfloat16, 0),
    (5, 3, 128, 128, [24, 20, 20], False, False, torch.bfloat16, 128),
    (5, 3, 128, 128, [24, 20, 20], False, True, torch.bfloat16, 128),
    (130, 5, 128, 64, [10, 12, 6, 4], True, True, torch.bfloat16, 64),
    (7, 4, 64, 64, [32], True, False, torch.float32, 0),
    (3, 2, 80, 36, [8, 10], False, False, torch.bfloat16, 3),     # one pair at a time
    (9, 1, 6, 2, None, False, False, torch.float32, 1),
    (4, 2, 96, 60, [10, 20], True, False, torch.bfloat16, 2),     # two pairs at a time
    (33, 2, 256, 256, [64, 64], False, False, torch.float32, 4),
    (2, 2, 512, 512, [256], False, False, torch.bfloat16, 0),
    (70, 64, 128, 128, None, False, False, torch.bfloat16, 4096),
    (600, 7, 64, 32, [0, 16], False, False, torch.bfloat16, 0),
    (11, 3, 64, 24, None, True, False, torch.bfloat16, 0),        # vectors that do not pair up
    (6, 2, 72, 48, None, False, False, torch.bfloat16, 0),
    (6, 2, 72, 64, [20, 12], True, True, torch.float32, 0),
    (3, 4096, 1024, 2, None, False, False, torch.bfloat16, 1),    # the most units in a row
])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(tokens, heads, d, rot, sections, adjacent, dealt, dtype, extra, inverse):
    g = gen(tokens + d)
    ld = heads * d + extra
    x = torch.randn(tokens, ld, generator=g).to(dtype).to(DEV)
    axes = len(sections) if sections else 1
    pos = torch.randint(-3, 5000, (axes, tokens), generator=g, dtype=torch.int32)
    pos[0, 0] = 2 ** 31 - 1
    pos[-1, -1] = -(2 ** 31)
    freq = torch.tensor([500000.0 ** (-2.0 * p / rot) for p in range(rot // 2)]).float()
    spec = L.make_rotary_spec(rot, sections, adjacent, dealt)
    ref = O.rotary(to_f64(x)[:, : heads * d].reshape(tokens, heads, d), pos.numpy(), freq.numpy(),
                   rot, sections or [rot // 2], adjacent, dealt, inverse).reshape(tokens, -1)
    call = L.mc_rotary_backward if inverse else L.mc_rotary_forward
    # one rounding of the result; the angle's 2^-24 of a turn and a 32-bit product and sum
    size = np.abs(to_f64(x)[:, : heads * d]).max()
    half = torch.finfo(dtype).eps / 2
    tol = half * np.abs(ref) + size * 2.0 ** -20
    out = torch.full((tokens + 1, heads * d + 5), 7.0, dtype=dtype, device=DEV)
    st = status()
    pd, fd = pos.to(DEV), freq.to(DEV)
    assert call(x, out, tokens, heads, d, ld, heads * d + 5, pd, fd, spec, st) == 0
    check_status(st)
    got = to_f64(out)
    assert (np.abs(got[:tokens, : heads * d] - ref) <= tol).all()
    assert (got[tokens:] == 7).all() and (got[:, heads * d:] == 7).all()
    # in place, at an address and stride that only whole elements divide
    y = torch.full((tokens * (ld + 1) + 1,), 7.0, dtype=dtype, device=DEV)
    rows = y[1:].view(tokens, ld + 1)
    rows[:, :ld] = x
    assert call(rows, rows, tokens, heads, d, ld + 1, ld + 1, pd, fd, spec, st) == 0
    check_status(st)
    assert torch.equal(rows[:, : heads * d], out[:tokens, : heads * d])
    assert torch.equal(rows[:, heads * d: ld], x[:, heads * d:]) and float(y[0]) == 7


def test_rotary_there_and_back():
    x = torch.randn(100, 4 * 128, generator=gen(3)).to(DEV)
    pos, freq = i32(np.arange(100)[None] + 10 ** 6), torch.rand(64, generator=gen(4)).to(DEV)
    spec = L.make_rotary_spec(128)
    y, z = torch.empty_like(x), torch.empty_like(x)
    assert L.mc_rotary_forward(x, y, 100, 4, 128, 512, 512, pos, freq, spec) == 0
    assert L.mc_rotary_backward(y, z, 100, 4, 128, 512, 512, pos, freq, spec) == 0
    assert float((z - x).abs().max()) < 8 * 2.0 ** -20


def test_rotary_offsets_past_32_bits():
    """Rows whose elements lie beyond 2^31: the last ones against the oracle."""
    tokens, ld = 70000, 32768
    x = torch.zeros(tokens, ld, dtype=torch.bfloat16, device=DEV)
    x[-3:, :256] = bf16(gen(8), 3, 256)
    pos, freq = i32(np.arange(tokens)[None]), torch.rand(64, generator=gen(9))
    want = O.rotary(to_f64(x[-3:, :256]).reshape(3, 2, 128), pos[:, -3:].cpu().numpy(),
                    freq.numpy(), 128, [64]).reshape(3, -1)
    tol = 2.0 ** -8 * np.abs(want) + np.abs(to_f64(x[-3:, :256])).max() * 2.0 ** -20
    st = status()
    assert L.mc_rotary_forward(x, x, tokens, 2, 128, ld, ld, pos, freq.to(DEV),
                               L.make_rotary_spec(128), st) == 0
    check_status(st)
    assert (np.abs(to_f64(x[-3:, :256]) - want) <= tol).all()
    assert not x[-3:, 256:].any() and not x[:-3].any()


# ------------------------------------------------------------------ masks
def make_documents(off, pre, causal, window, b, s):
    n = 2 * b * ((s + 127) // 128)
    lo = torch.full((b * s + 1,), -7, dtype=torch.int32, device=DEV)
    hi = torch.full((b * s + 1,), -7, dtype=torch.int32, device=DEV)
    tab = torch.full((n * 4 + 1,), -7, dtype=torch.int32, device=DEV)
    assert L.mc_attention_mask_table_ints(b, s) == 4 * n
    st = status()
    assert L.mc_attention_mask_documents(i32(off), len(off) - 1, None if pre is None else i32(pre),
                                         int(causal), window, b, s, lo, hi, tab, st) == 0
    check_status(st)
    assert int(lo[-1]) == int(hi[-1]) == int(tab[-1]) == -7
    return lo[:-1].view(b, s), hi[:-1].view(b, s), tab[:-1]


def table_lists(tab):
    rows = [tuple(r) for r in tab.view(2, -1, 4)[0].tolist()], \
        [tuple(r) for r in tab.view(2, -1, 4)[1].tolist()]
    return rows


@pytest.mark.parametrize("off,pre,causal,window,b,s", [
    ([0, 1], None, True, 0, 1, 1),
    ([0, 128], None, True, 0, 1, 128),
    ([5, 9, 9, 9, 200, 300], [1, 0, 0, -1, 50], True, 0, 1, 310),
    ([0, 700], None, True, 0, 2, 350),                 # one document over both sequences
    ([0, 100, 450, 700], [30, 100, 1000], True, 0, 2, 350),
    ([0, 100, 450, 700], [30, 100, 1000], True, 17, 2, 350),
    ([0, 100, 450, 700], None, False, 0, 2, 350),
    ([0, 100, 450, 700], None, False, 1, 2, 350),
    ([0], None, True, 0, 2, 140),                      # no documents
    (list(range(0, 261)), None, True, 0, 1, 260),      # a document per token
    ([0] * 300 + [50] * 300 + [64], None, True, 0, 1, 70),   # hundreds of empty ones
    ([0, 512], None, True, 2 ** 31 - 1, 1, 512),
    ([-5, 60], None, True, 0, 1, 70),
])
def test_mask_documents(off, pre, causal, window, b, s):
    lo, hi, tab = make_documents(off, pre, causal, window, b, s)
    rlo, rhi = O.document_intervals(off, pre, causal, window, b, s)
    assert lo.cpu().tolist() == rlo.tolist() and hi.cpu().tolist() == rhi.tolist()
    q, k = table_lists(tab)
    rq, rk = O.tables(rlo, rhi)
    assert q == rq and k == rk


@pytest.mark.parametrize("b,s", [(1, 900), (3, 257), (40, 130)])
def test_mask_intervals_any(b, s):
    g = np.random.default_rng(s)
    lo, hi = g.integers(-20, s + 20, (b, s)), g.integers(-20, s + 20, (b, s))
    lo[:, 130:260], hi[:, 130:260] = 5, 5
    tab = torch.empty(L.mc_attention_mask_table_ints(b, s), dtype=torch.int32, device=DEV)
    st = status()
    assert L.mc_attention_mask_intervals(b, s, i32(lo), i32(hi), tab, st) == 0
    check_status(st)
    assert table_lists(tab) == O.tables(lo, hi)


def test_mask_tables_of_many_blocks():
    """More entries than are sorted: the sequence's order, query blocks backwards."""
    b, s = 4200, 7
    off = list(range(0, b * s + 1, 7))
    lo, hi, tab = make_documents(off, None, True, 0, b, s)
    q, k = table_lists(tab)
    assert q == [(x, 0, 0, 7) for x in reversed(range(b))] and k == [(x, 0, 0, 1) for x in range(b)]
    assert (lo == 0).all() and (hi == torch.arange(1, 8, device=DEV)).all()
    b, s = 2, 300000
    lo, hi, tab = make_documents([0, 600000], None, True, 0, b, s)
    nb = (s + 127) // 128
    q, k = table_lists(tab)
    assert q[0] == (1, nb - 1, 0, s) and q[-1] == (0, 0, 0, 128)
    assert k[0] == (0, 0, 0, nb) and k[nb + 3] == (1, 3, 3, nb)


@pytest.mark.parametrize("b,s,docs", [(7, 5000, 9000), (1, 40000, 33), (300, 257, 1500)])
def test_mask_tables_over_several_turns(b, s, docs):
    """More blocks than a cluster forms at once, and searches of several rounds."""
    g = torch.Generator().manual_seed(docs)
    cuts = torch.randint(0, b * s - 4, (docs - 1,), generator=g).sort().values.tolist()
    off = [0] + cuts + [b * s - 5]
    pre = torch.randint(-1, 40, (docs,), generator=g).tolist()
    lo, hi, tab = make_documents(off, pre, True, 900, b, s)
    rlo, rhi = O.document_intervals(off, pre, True, 900, b, s)
    assert lo.cpu().tolist() == rlo.tolist() and hi.cpu().tolist() == rhi.tolist()
    q, k = table_lists(tab)
    rq, rk = O.tables(rlo, rhi)
    assert q == rq and k == rk


# ------------------------------------------------------------------ attention
def random_intervals(b, s, seed):
    """Intervals with no order, some empty, some past the sequence's ends."""
    g = np.random.default_rng(seed)
    lo = g.integers(-5, s + 1, (b, s))
    hi = lo + g.integers(-3, max(2, s // 2), (b, s))
    return lo, hi


def intervals(kind, b, s):
    if kind == "causal":
        return O.document_intervals([x * s for x in range(b + 1)], None, True, 0, b, s)
    if kind == "documents":
        cuts = sorted({0, b * s - min(9, s // 2), *[(k * 97) % (b * s) for k in range(1, 6)]})
        return O.document_intervals(cuts, None, True, 0, b, s)
    if kind == "prefix":
        cuts = sorted({0, b * s, *[(k * 131) % (b * s) for k in range(1, 4)]})
        return O.document_intervals(cuts, [60] * (len(cuts) - 1), True, 0, b, s)
    if kind == "window":
        return O.document_intervals([x * s for x in range(b + 1)], None, True, 70, b, s)
    if kind == "whole":
        return O.document_intervals([x * s for x in range(b + 1)], None, False, 0, b, s)
    if kind == "any":
        return random_intervals(b, s, s)
    assert kind == "nothing"
    return np.zeros((b, s), dtype=np.int64), np.zeros((b, s), dtype=np.int64)


class Problem:
    """One attention problem on the GPU, and its oracle."""

    def __init__(self, kind, b, s, H, d, cap=0.0, bias=False, qstd=1.0, seed=0):
        g = gen(seed + s)
        self.b, self.s, self.H, self.d, self.cap = b, s, H, d, cap
        a = H * d
        qkv = torch.randn(b, s, 3 * a, generator=g)
        qkv[:, :, :a] *= qstd
        self.qkv = qkv.bfloat16().to(DEV)
        self.dout = bf16(g, b, s, a)
        self.lo, self.hi = intervals(kind, b, s)
        self.slopes = [2.0 ** -(k + 1) for k in range(H)] if bias else None
        self.causal = bool(np.all(np.minimum(self.hi, s) <= np.arange(1, s + 1)[None]))
        self.klo, self.khi = i32(self.lo), i32(self.hi)
        self.tab = torch.empty(L.mc_attention_mask_table_ints(b, s), dtype=torch.int32, device=DEV)
        self.sl = None if not bias else torch.tensor(self.slopes, device=DEV)
        assert L.mc_attention_mask_intervals(b, s, self.klo, self.khi, self.tab) == 0
        self.opt = L.make_attention_options(self.klo, self.khi, self.tab, self.sl, cap, self.causal)
        self.o = torch.full((b * s + 1, a), 3.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((b * H * s + 1,), 3.0, device=DEV)
        self.delta = torch.empty(b * H * s, device=DEV)

    def forward(self, stream=None):
        st = status()
        assert L.mc_attention_forward_opt(self.qkv, self.o, self.lse, self.b, self.s, self.H,
                                          self.d, self.opt, st, stream) == 0
        check_status(st)
        assert (self.o[-1] == 3).all() and float(self.lse[-1]) == 3
        return (to_f64(self.o[:-1]).reshape(self.b, self.s, -1),
                to_f64(self.lse[:-1]).reshape(self.b, self.H, self.s))

    def backward(self, tiles):
        b, s, H, d = self.b, self.s, self.H, self.d
        dqkv = torch.full((b * s + 1, 3 * H * d), 3.0, dtype=torch.bfloat16, device=DEV)
        n = L.mc_attention_backward_opt_ws_bytes(b, s, H, d, self.opt) if tiles else 0
        ws = torch.full((n + 256,), 0xff, dtype=torch.uint8, device=DEV) if tiles else None  # NaN
        st = status()
        assert L.mc_attention_backward_opt(self.qkv, self.o, self.lse, self.dout, dqkv, self.delta,
                                           b, s, H, d, self.opt, ws, n, st) == 0
        check_status(st)
        assert (dqkv[-1] == 3).all()
        if tiles:
            assert (ws[n:] == 0xff).all()
        return to_f64(dqkv[:-1]).reshape(b, s, -1)

    def check(self, tiles=(False, True)):
        qkv, dout = to_f64(self.qkv), to_f64(self.dout)
        o, lse, tol, ltol = O.attention_forward(qkv, self.lo, self.hi, self.H, self.d, self.slopes,
                                                self.cap)
        got, glse = self.forward()
        off = np.abs(got - o) / tol
        assert off.max() <= 1, f"O: {off.max():.3g} of the tolerance"
        seen = np.isfinite(lse)
        assert np.array_equal(glse[~seen], lse[~seen])
        if seen.any():
            off = np.abs(glse - lse)[seen] / ltol[seen]
            assert off.max() <= 1, f"lse: {off.max():.3g} of the tolerance"
        ref, tol, tol32 = O.attention_backward(qkv, dout, self.lo, self.hi, self.H, self.d, self.slopes,
                                        self.cap)
        a = self.H * self.d
        for t in tiles:
            got = self.backward(t)
            for n, name in enumerate(("dQ", "dK", "dV")):
                c = slice(n * a, (n + 1) * a)
                off = np.abs(got - ref)[..., c] / tol[..., c]
                assert off.max() <= 1, f"{name}, tiles {t}: {off.max():.3g} of the tolerance"
                norm = np.linalg.norm(ref[..., c])
                # Roundings of either sign: the 2-norm within two of them, and the
                # 32-bit part: with one visible key dz = P (dP - delta) is the
                # difference of the same d products summed in two orders, up to
                # d 2^-24 of their size each, and no bf16 step of 0 covers that.
                assert np.linalg.norm((got - ref)[..., c]) <= \
                    2 * O.HALF_BF16 * norm + np.linalg.norm(tol32[..., c]), name


@pytest.mark.parametrize("s", [1, 2, 63, 64, 127, 128, 129, 255, 256, 257, 400])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_lengths(s, d):
    Problem("causal", 1, s, 2, d).check()


@pytest.mark.parametrize("kind", ["documents", "prefix", "window", "whole", "any", "nothing"])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (4.0, False), (0.0, True), (4.0, True)])
@pytest.mark.parametrize("b,s,H,d", [(2, 333, 2, 128), (1, 450, 3, 64)])
def test_attention_masks_and_scores(kind, cap, bias, b, s, H, d):
    Problem(kind, b, s, H, d, cap, bias, qstd=2.0 if cap else 1.0).check()


@pytest.mark.parametrize("kind", ["documents", "any"])
def test_attention_one_row_and_many_sequences(kind):
    Problem(kind, 37, 1, 3, 64, 5.0, True).check()
    Problem(kind, 19, 11, 1, 128).check()


def test_attention_thousands_of_short_sequences():
    """More table entries than are sorted, a few rows in each block."""
    Problem("any", 4500, 3, 2, 64, 5.0, True).check(tiles=(True,))


def test_attention_many_blocks():
    """More CTAs than four waves: the grid goes head after head."""
    Problem("window", 6, 1200, 12, 64).check()


@pytest.mark.parametrize("where", ["front", "back", "both"])
def test_attention_many_empty_blocks(where):
    """Long padding: a CTA's share is one block with keys among many without."""
    p = Problem("causal", 1, 4000, 40, 64)
    lo, hi = p.lo.copy(), p.hi.copy()
    if where == "front":
        lo[:, 100:], hi[:, 100:] = 0, 0
    elif where == "back":
        lo[:, :3900], hi[:, :3900] = 0, 0
    else:
        lo[:, 100:3900], hi[:, 100:3900] = 0, 0
    seen = lo[0] < hi[0]
    lo[:, 3900:] = np.where(lo[:, 3900:] < hi[:, 3900:], 3900, 0)
    p.klo.copy_(i32(lo))
    p.khi.copy_(i32(hi))
    assert L.mc_attention_mask_intervals(1, 4000, p.klo, p.khi, p.tab) == 0
    o, lse = p.forward()
    assert (o[0, ~seen] == 0).all() and (lse[0][:, ~seen] == -np.inf).all()
    d = [p.backward(t) for t in (False, True)]
    # the two ends are independent short sequences
    for at, n in ((0, 100), (3900, 100)):
        if not seen[at]:
            continue
        q = Problem("causal", 1, n, 40, 64)
        q.qkv.copy_(p.qkv[:, at:at + n])
        q.dout.copy_(p.dout[:, at:at + n])
        o2, lse2 = q.forward()
        assert np.abs(lse[0][:, at:at + n] - lse2[0]).max() < 1e-4
        assert np.linalg.norm(o[0, at:at + n] - o2[0]) <= 2 * O.HALF_BF16 * np.linalg.norm(o2)
        for t in (False, True):
            d2 = q.backward(t)
            assert np.linalg.norm(d[t][0, at:at + n] - d2[0]) <= \
                2 * O.HALF_BF16 * np.linalg.norm(d2)
            rest = d[t][0, ~seen]
            assert (rest == 0).all()


def test_attention_scores_far_beyond_the_cap():
    # scores of several hundred against a cap of 2: the cap's derivative is 0, nothing overflows
    Problem("documents", 1, 200, 2, 64, cap=2.0, qstd=300.0).check()


def test_attention_large_scores_and_steep_bias():
    p = Problem("causal", 1, 300, 2, 128, bias=True, qstd=20.0)
    p.sl.mul_(64.0)
    p.slopes = [64.0 * x for x in p.slopes]
    p.check()


@pytest.mark.parametrize("kind", ["causal", "window", "whole"])
@pytest.mark.parametrize("cap,d", [(0.0, 128), (0.0, 64), (5.0, 64)])
def test_attention_slopes_of_both_signs(kind, cap, d):
    p = Problem(kind, 1, 430, 3, d, cap, True)
    p.slopes = [-0.125, 0.0, 0.25]  # negative: far keys count more
    p.sl.copy_(torch.tensor(p.slopes))
    p.check()


@pytest.mark.parametrize("cap", [2.0 ** -16, 0.01, 5000.0, 2.0 ** 16])
def test_attention_smallest_and_largest_caps(cap):
    p = Problem("documents", 1, 333, 2, 64, cap, qstd=2.0)
    p.qkv[:, 200:, :128] = 0  # scores of 0 too
    if cap == 2.0 ** 16:
        # c tanh(z / c) is z - z^3 / (3 c^2): for |z| < 40 that is z to within 5e-6, below the
        # tolerance without a cap (which has no term in c)
        p.cap = 0.0
    p.check()


def test_matches_plain_causal_attention():
    p = Problem("causal", 2, 777, 4, 128)
    o, lse = p.forward()
    o2 = torch.empty(2 * 777, 512, dtype=torch.bfloat16, device=DEV)
    lse2 = torch.empty(2 * 4 * 777, device=DEV)
    assert L.mc_attention_forward(p.qkv, o2, lse2, 2, 777, 4, 128) == 0
    # both within two roundings (P and O) of the same values
    assert np.linalg.norm(o - to_f64(o2).reshape(o.shape)) <= 4 * O.HALF_BF16 * np.linalg.norm(o)
    assert np.abs(lse - to_f64(lse2).reshape(lse.shape)).max() < 1e-5 * 10
    for tiles in (False, True):
        d = p.backward(tiles)
        d2 = torch.empty(2 * 777, 1536, dtype=torch.bfloat16, device=DEV)
        assert L.mc_attention_backward(p.qkv, o2, lse2, p.dout, d2, p.delta, 2, 777, 4, 128) == 0
        assert np.linalg.norm(d - to_f64(d2).reshape(d.shape)) <= \
            4 * O.HALF_BF16 * np.linalg.norm(d)


def test_attention_is_repeatable_and_unseen_rows_have_no_influence():
    p = Problem("documents", 1, 600, 4, 128, cap=10.0, qstd=2.0)
    o, lse = p.forward()
    d = [p.backward(t) for t in (False, True)]
    pad = np.nonzero(p.lo[0] >= p.hi[0])[0]
    assert len(pad) == 9
    p.qkv[0, pad[0]:] = 1e30
    p.dout[0, pad[0]:] = -1e4
    o2, lse2 = p.forward()
    assert np.array_equal(o, o2) and np.array_equal(lse, lse2)
    for t in (False, True):
        d2 = p.backward(t)
        assert np.array_equal(d[t], d2) and (d2[0, pad[0]:] == 0).all()


def test_nan_is_not_hidden():
    p = Problem("causal", 1, 300, 1, 64)
    p.qkv[0, 40, 0] = math.nan        # a query
    o, lse = p.forward()
    assert np.isnan(o[0, 40]).all() and np.isnan(lse[0, 0, 40])
    rest = np.delete(o[0], 40, axis=0)
    assert np.isfinite(rest).all()


def test_interval_past_its_query_is_reported():
    """causal = True with intervals that look ahead: an error status, no store
    outside the smaller workspace."""
    p = Problem("whole", 1, 400, 2, 64)
    p.forward()
    p.opt.causal = 1
    n = L.mc_attention_backward_opt_ws_bytes(1, 400, 2, 64, p.opt)
    ws = torch.full((n + 65536,), 0x55, dtype=torch.uint8, device=DEV)
    dqkv = torch.empty(400, 384, dtype=torch.bfloat16, device=DEV)
    st = status()
    assert L.mc_attention_backward_opt(p.qkv, p.o, p.lse, p.dout, dqkv, p.delta, 1, 400, 2, 64,
                                       p.opt, ws, n, st) == 0
    torch.cuda.synchronize()
    assert int(st[0]) == L.MC_ERR_DEVICE_BOUNDS and (ws[n:] == 0x55).all()


def test_tables_of_another_shape_are_reported():
    p = Problem("causal", 1, 400, 2, 64)
    p.tab[0] = 3        # a sequence that is not there
    st = status()
    assert L.mc_attention_forward_opt(p.qkv, p.o, p.lse, 1, 400, 2, 64, p.opt, st) == 0
    torch.cuda.synchronize()
    assert int(st[0]) == L.MC_ERR_DEVICE_BOUNDS


def windowed_tail_matches(qkv, o, dqkv, dout, lo, hi, H, d, window, n=320):
    """The last rows of the last head of the last sequence, which only depend on
    the n tokens that end it."""
    a, b, s = H * d, qkv.shape[0], qkv.shape[1]
    part = lambda x, k: x[b - 1:, s - n:, k * a + (H - 1) * d:k * a + H * d]  # noqa: E731
    sub = to_f64(torch.cat([part(qkv, k) for k in range(3)], dim=2))
    slo, shi = ((v[b - 1:, s - n:].cpu().numpy() - (s - n)).clip(0, n) for v in (lo, hi))
    want, _, tol, _ = O.attention_forward(sub, slo, shi, 1, d)
    assert (np.abs(to_f64(part(o, 0)) - want) <= tol)[:, window:].all()
    want, tol, _ = O.attention_backward(sub, to_f64(part(dout, 0)), slo, shi, 1, d)
    got = to_f64(torch.cat([part(dqkv, k) for k in range(3)], dim=2))
    assert (np.abs(got - want) <= tol)[:, window:].all()


@pytest.mark.parametrize("b,s,H,d,tiles", [(1, 100000, 64, 128, False), (2, 50000, 64, 128, False),
                                           (1, 16500, 18, 64, True)])
def test_attention_offsets_past_32_bits(b, s, H, d, tiles):
    """Elements beyond 2^31 in Q | K | V, or tiles beyond 2^32 bytes."""
    a, window = H * d, 64
    qkv, dqkv = (torch.empty(b, s, 3 * a, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    o, dout = (torch.empty(b, s, a, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    torch.manual_seed(s)
    qkv.normal_()
    dout.normal_()
    lse, delta = (torch.empty(b * H * s, device=DEV) for _ in range(2))
    lo, hi, tab = make_documents([0, b * s - s // 2, b * s], None, True, window, b, s)
    opt = L.make_attention_options(lo, hi, tab)
    n = L.mc_attention_backward_opt_ws_bytes(b, s, H, d, opt) if tiles else 0
    assert not tiles or n > 2 ** 32
    ws, st = torch.empty(n, dtype=torch.uint8, device=DEV) if tiles else None, status()
    assert L.mc_attention_forward_opt(qkv, o, lse, b, s, H, d, opt, st) == 0
    assert L.mc_attention_backward_opt(qkv, o, lse, dout, dqkv, delta, b, s, H, d, opt, ws, n,
                                       st) == 0
    check_status(st)
    windowed_tail_matches(qkv, o, dqkv, dout, lo, hi, H, d, window)


def test_two_streams_at_once_give_the_same_bits():
    """Grids of more items than start at once, whose CTAs take items as they come."""
    ps = [Problem("documents", 1, 2500, 40, 128, 30.0, seed=1),
          Problem("window", 2, 1100, 40, 64, bias=True, seed=2)]
    n = [L.mc_attention_backward_opt_ws_bytes(p.b, p.s, p.H, p.d, p.opt) for p in ps]
    ws = [torch.empty(x, dtype=torch.uint8, device=DEV) for x in n]
    out = [torch.empty_like(p.qkv) for p in ps]
    st = [status(), status()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def call(i, stream):
        p = ps[i]
        assert L.mc_attention_forward_opt(p.qkv, p.o, p.lse, p.b, p.s, p.H, p.d, p.opt, st[i],
                                          stream) == 0
        assert L.mc_attention_backward_opt(p.qkv, p.o, p.lse, p.dout, out[i], p.delta, p.b, p.s,
                                           p.H, p.d, p.opt, ws[i], n[i], st[i], stream) == 0

    for i in range(2):
        call(i, None)
    torch.cuda.synchronize()
    alone = [(p.o.clone(), p.lse.clone(), x.clone()) for p, x in zip(ps, out)]
    for p, x in zip(ps, out):
        p.o.zero_(), p.lse.zero_(), x.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            call(i, streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        check_status(st[i])
        p = ps[i]
        rows = p.b * p.s
        assert torch.equal(p.o[:rows], alone[i][0][:rows])
        assert torch.equal(p.lse[:-1], alone[i][1][:-1]) and torch.equal(out[i], alone[i][2])


def test_two_graphs_share_a_workspace():
    ps = [Problem("documents", 1, 700, 4, 64, seed=1), Problem("prefix", 2, 300, 3, 128, seed=2)]
    n = [L.mc_attention_backward_opt_ws_bytes(p.b, p.s, p.H, p.d, p.opt) for p in ps]
    ws = torch.empty(max(n), dtype=torch.uint8, device=DEV)
    out, graphs, alone = [torch.empty_like(p.qkv) for p in ps], [], []
    stream = torch.cuda.Stream()
    for i, p in enumerate(ps):
        def call(i=i, p=p):
            assert L.mc_attention_forward_opt(p.qkv, p.o, p.lse, p.b, p.s, p.H, p.d, p.opt, None,
                                              stream) == 0
            assert L.mc_attention_backward_opt(p.qkv, p.o, p.lse, p.dout, out[i], p.delta, p.b, p.s,
                                               p.H, p.d, p.opt, ws, n[i], None, stream) == 0
        with torch.cuda.stream(stream):
            call()
        torch.cuda.synchronize()
        alone.append(out[i].clone())
        out[i].zero_()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            call()
        graphs.append(g)
    for i in (0, 1, 1, 0, 0, 1):
        out[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(out[i], alone[i])


def test_on_a_stream_and_in_a_graph():
    """Mask, rotary, attention and its backward captured together and replayed
    on new documents and values."""
    b, s, H, d = 1, 300, 2, 64
    a = H * d
    qkv = torch.zeros(b * s, 3 * a, dtype=torch.bfloat16, device=DEV)
    dout = bf16(gen(5), b, s, a)
    off, pos = i32([0, 100, 300]), i32(np.arange(s)[None])
    freq = torch.rand(32, generator=gen(6)).to(DEV)
    lo, hi = (torch.empty(b, s, dtype=torch.int32, device=DEV) for _ in range(2))
    tab = torch.empty(L.mc_attention_mask_table_ints(b, s), dtype=torch.int32, device=DEV)
    opt = L.make_attention_options(lo, hi, tab, softcap=20.0)
    o, lse = torch.empty(b * s, a, dtype=torch.bfloat16, device=DEV), torch.empty(H * s, device=DEV)
    dqkv, delta = torch.empty_like(qkv), torch.empty(H * s, device=DEV)
    n = L.mc_attention_backward_opt_ws_bytes(b, s, H, d, opt)
    ws, st = torch.empty(n, dtype=torch.uint8, device=DEV), status()
    spec = L.make_rotary_spec(64, [16, 16][:1] + [16], interleaved_axes=True)
    pos2 = torch.cat([pos, pos * 3]).contiguous()

    def step(stream):
        rc = [L.mc_attention_mask_documents(off, 2, None, 1, 0, b, s, lo, hi, tab, st, stream),
              L.mc_rotary_forward(qkv, qkv, b * s, 2 * H, d, 3 * a, 3 * a, pos2, freq, spec, st, stream),
              L.mc_attention_forward_opt(qkv, o, lse, b, s, H, d, opt, st, stream),
              L.mc_attention_backward_opt(qkv, o, lse, dout, dqkv, delta, b, s, H, d, opt, ws, n, st,
                                          stream),
              L.mc_rotary_backward(dqkv, dqkv, b * s, 2 * H, d, 3 * a, 3 * a, pos2, freq, spec, st,
                                   stream)]
        assert rc == [0] * 5

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for seed, cut in ((1, 100), (2, 17), (3, 299)):
        x = bf16(gen(seed), b * s, 3 * a)
        off.copy_(i32([0, cut, 300]))
        qkv.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        check_status(st)
        got = [t.clone() for t in (o, lse, dqkv)]
        qkv.copy_(x)
        step(torch.cuda.current_stream())
        torch.cuda.synchronize()
        for u, v in zip(got, (o, lse, dqkv)):
            assert torch.equal(u, v)


# ------------------------------------------------------------------ the layer
def torch_layer(x, w, H, d, tokens_of, rot, lo, hi, slopes, cap):
    """The layer in torch float64 on the CPU, rotary and mask in the attention."""
    b, s, h = x.shape
    a = H * d
    ln = lambda v, g, c: torch.nn.functional.layer_norm(v, (h,), g, c, 1e-5)  # noqa: E731
    qkv = ln(x, w["ln1_g"], w["ln1_b"]) @ w["w_qkv"].T + w["b_qkv"]
    q, k, v = (t.reshape(b, s, H, d).transpose(1, 2) for t in qkv.split(a, dim=-1))
    if rot is not None:
        rd, axes, pos, freq = rot
        ang = torch.stack([pos[axes[p]].double() * float(freq[p]) for p in range(rd // 2)], -1)
        cos, sin = torch.cos(ang).view(b, 1, s, -1), torch.sin(ang).view(b, 1, s, -1)

        def turn(t):
            u, z, rest = t[..., : rd // 2], t[..., rd // 2: rd], t[..., rd:]
            return torch.cat([u * cos - z * sin, u * sin + z * cos, rest], -1)
        q, k = turn(q), turn(k)
    z = q @ k.transpose(-1, -2) / math.sqrt(d)
    if cap:
        z = cap * torch.tanh(z / cap)
    i = torch.arange(s)
    if slopes is not None:
        z = z - torch.tensor(slopes).double()[:, None, None] * (i[:, None] - i[None]).abs()
    seen = (i >= lo[:, None, :, None]) & (i < hi[:, None, :, None])
    z = z.masked_fill(~seen, -1e300)
    p = torch.softmax(z, -1) * seen
    o = (p @ v).transpose(1, 2).reshape(b, s, a)
    x1 = x + o @ w["w_o"].T + w["b_o"]
    u = ln(x1, w["ln2_g"], w["ln2_b"]) @ w["w_fc1"].T + w["b_fc1"]
    u = torch.nn.functional.gelu(u, approximate="tanh")
    return x1 + u @ w["w_fc2"].T + w["b_fc2"]


@pytest.mark.parametrize("flags", [dict(), dict(recompute=True), dict(sequence_parallel=True),
                                   dict(attn_dq_recompute=True), dict(fp8=True)])
@pytest.mark.parametrize("ahead", [False, True])
def test_layer_with_positions_and_mask(flags, ahead):
    from megatron_transformer_layer_gb300.layer import TransformerLayer
    from parity import assert_close
    b, s, h, H, f = 2, 152, 256, 4, 512
    d, T = 64, 2 * 152
    g = gen(11)
    params = TransformerLayer.random_params(h, H, f, seed=3, std=0.05)
    for n in ("b_qkv", "b_o", "b_fc1", "b_fc2", "ln1_b", "ln2_b"):
        params[n] = bf16(g, params[n].numel(), std=0.1)
    off, pre = [0, 40, 152, 250, 300], [10, 30, 0, 20] if ahead else None
    lo, hi, tab = make_documents(off, pre, True, 0, b, s)
    slopes = torch.tensor([0.5, 0.25, 0.125, 0.0625], device=DEV)
    att = L.make_attention_options(lo, hi, tab, slopes, 8.0, causal=not ahead)
    pos = torch.randint(0, 400, (2, T), generator=g, dtype=torch.int32)
    freq = torch.rand(24, generator=g)
    pd, fd = pos.to(DEV), freq.to(DEV)
    rot = L.make_layer_rotary(L.make_rotary_spec(48, [16, 8], interleaved_axes=True), pd, fd)
    layer = TransformerLayer(b, s, h, H, f, 2, params=params, rotary=rot, attention=att, **flags)
    x = torch.randn(T, h, generator=g).to(DEV)
    dy = torch.randn(T, h, generator=g).to(DEV)
    y = layer.forward(x)
    dx = layer.backward(dy)
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    w = {n: v.detach().double().cpu().requires_grad_() for n, v in params.items()}
    x64 = x.double().cpu().view(b, s, h).requires_grad_()
    axes = O.axis_of_pair([16, 8], dealt=True)
    y64 = torch_layer(x64, w, H, d, None, (48, axes, pos, freq), lo.cpu().long(), hi.cpu().long(),
                      slopes.tolist(), 8.0)
    y64.backward(dy.double().cpu().view(b, s, h))
    # The layer's own gate (bf16).  FP8: a gradient goes through up to two chained
    # products whose E5M2 operand is off by at most 2^-3 of itself, so a sum of n
    # terms of either sign, sqrt(n) terms large, is off by up to 2 * 2^-3 sqrt(n)
    # terms: 2^-2 of its own size, which is at most max|o| for the largest error
    # and, as mean|o| is about a quarter of max|o|, 2^-4 of max|o| on average.
    tol = (2e-2, 2e-3) if not flags.get("fp8") else (2.0 ** -2, 2.0 ** -4)
    assert_close("y", to_f64(y), y64.detach().numpy().reshape(T, h), *tol)
    assert_close("dx", to_f64(dx), x64.grad.numpy().reshape(T, h), *tol)
    for n in w:
        assert_close(n, to_f64(layer.grads[n]), w[n].grad.numpy(), *tol)


def test_layer_without_them_is_unchanged():
    from megatron_transformer_layer_gb300.layer import TransformerLayer
    params = TransformerLayer.random_params(256, 4, 512, seed=5)
    x, dy = torch.randn(200, 256, generator=gen(1)).to(DEV), torch.randn(200, 256, generator=gen(2)).to(DEV)
    layer = TransformerLayer(1, 200, 256, 4, 512, params=params)
    y, dx = layer.forward(x), layer.backward(dy)
    grads = {k: v.clone() for k, v in layer.grads.items()}
    y2, dx2 = torch.empty_like(y), torch.empty_like(dx)
    assert L.mc_layer_forward(layer.shape, layer.weights, x, y2, layer.saved, layer.ws,
                              layer.ws_bytes, torch.cuda.current_stream()) == 0
    assert L.mc_layer_backward(layer.shape, layer.weights, x, dy, layer.saved, dx2,
                               ctypes.cast(ctypes.pointer(layer._grads_c),
                                           ctypes.POINTER(L.mc_layer_grads)).contents,
                               layer.ws, layer.ws_bytes, torch.cuda.current_stream()) == 0
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(dx, dx2)
    for k in grads:
        assert torch.equal(grads[k], layer.grads[k])
