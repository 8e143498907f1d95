"""Attention to keys of another length and the norms of queries and keys, without a
GPU: the float64 oracle against plainer forms and differences, workspace sizes, and
what the entry points and the binding refuse before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.cross_attention as O
from megatron_transformer_layer_gb300 import _lib as L

P = 1 << 20  # a pointer that is aligned and never dereferenced


# ------------------------------------------------------------------ the oracle
def problem(seed=1):
    g = np.random.default_rng(seed)
    heads, kv, d = 4, 2, 3
    q_seq = O.sequence_rows(3, 9, [0, 4, 5, 8], [3, 1, 3])
    k_seq = O.sequence_rows(3, 12, [1, 6, 6, 11], [5, 0, 4])
    q, k, v = (g.standard_normal((r, h * d)) for r, h in ((9, heads), (12, kv), (12, kv)))
    return g, (q, k, v), q_seq, k_seq, (heads, kv, d, 0.7)


def test_sequence_rows():
    assert O.sequence_rows(2, 8) == [(0, 4, 4), (4, 4, 4)]
    assert O.sequence_rows(2, 8, [2, 3, 99], [5, 5]) == [(2, 1, 1), (3, 5, 5)]
    assert O.sequence_rows(2, 8, [-4, 6, 1], [-1, 7]) == [(0, 6, 0), (6, 0, 0)]


def test_forward_oracle_by_loops():
    _, (q, k, v), q_seq, k_seq, (heads, kv, d, scale) = problem()
    o, lse, _, _, owned = O.forward(q, k, v, q_seq, k_seq, heads, kv, d, scale)
    for (q0, slot, nq), (k0, _, nk) in zip(q_seq, k_seq):
        for i in range(q0, q0 + slot):
            assert owned[i]
            for h in range(heads):
                g = h * kv // heads
                e = [np.exp(scale * q[i, h * d: h * d + d] @ k[j, g * d: g * d + d])
                     for j in range(k0, k0 + nk)] if i < q0 + nq else []
                for c in range(d):
                    want = sum(w * v[k0 + j, g * d + c] for j, w in enumerate(e)) / sum(e) if e else 0
                    assert np.isclose(o[i, h * d + c], want, atol=1e-13)
                assert np.isclose(lse[h, i], np.log(sum(e))) if e else lse[h, i] == -np.inf
    assert owned.sum() == 8 and not owned[8]


def test_backward_oracle_against_differences():
    g, qkv, q_seq, k_seq, a = problem(2)
    dout = g.standard_normal(qkv[0].shape)
    for (q0, slot, nq) in q_seq:
        dout[q0 + nq: q0 + slot] = 0
    got, _, _ = O.backward(*qkv, dout, q_seq, k_seq, *a)
    loss = lambda xs: (O.forward(*xs, q_seq, k_seq, *a)[0] * dout).sum()  # noqa: E731
    for n in range(3):
        for at in np.ndindex(qkv[n].shape):
            xs = [x.copy() for x in qkv]
            xs[n][at] += 1e-5
            up = loss(xs)
            xs[n][at] -= 2e-5
            assert abs((up - loss(xs)) / 2e-5 - got[n][at]) < 1e-8


TURN = (np.array([[3, -2, 70]]), np.array([0.5, 0.01], dtype=np.float32), 4, [2])


@pytest.mark.parametrize("centred", [False, True])
@pytest.mark.parametrize("turn", [None, TURN])
def test_norm_oracle_against_differences(centred, turn):
    g = np.random.default_rng(3)
    x, dout = g.standard_normal((3, 3, 5)), g.standard_normal((3, 3, 5))
    gains = [g.standard_normal(5) for _ in range(2)]
    shifts = [g.standard_normal(5) for _ in range(2)]
    loss = lambda x, gs, cs: (O.qk_norm(x, 2, 1, 1e-2, centred, gs, cs, turn) * dout).sum()  # noqa: E731
    dx, size, ((gq, gk), (cq, ck)) = O.qk_norm_backward(x, dout, 2, 1, 1e-2, centred, gains, turn)
    assert (np.abs(dx) <= size * (1 + 1e-12)).all()

    def slope(of, call):
        out = np.zeros_like(of)
        for at in np.ndindex(of.shape):
            y = of.copy()
            y[at] += 1e-5
            up = call(y)
            y[at] -= 2e-5
            out[at] = (up - call(y)) / 2e-5
        return out
    assert np.abs(slope(x, lambda y: loss(y, gains, shifts)) - dx).max() < 1e-8
    for i, (a, b) in enumerate(((gq, cq), (gk, ck))):
        put = lambda v, y: [y if j == i else v[j] for j in range(2)]  # noqa: E731
        assert np.abs(slope(gains[i], lambda y: loss(x, put(gains, y), shifts)) - a[0]).max() < 1e-8
        assert np.abs(slope(shifts[i], lambda y: loss(x, gains, put(shifts, y))) - b[0]).max() < 1e-8


def test_norm_oracle_is_torchs():
    g = np.random.default_rng(4)
    x, w, b = g.standard_normal((4, 2, 6)), g.standard_normal(6), g.standard_normal(6)
    want = torch.nn.functional.layer_norm(*map(torch.from_numpy, (x,)), (6,), torch.from_numpy(w),
                                          torch.from_numpy(b), 1e-3).numpy()
    assert np.allclose(O.qk_norm(x, 1, 1, 1e-3, True, (w, w), (b, b)), want, atol=1e-13)


# ------------------------------------------------------------------ sizes
def cross(**kw):
    a = dict(sequences=2, q_rows=200, kv_rows=300, heads=4, kv_heads=2, head_dim=64)
    a.update(kw)
    return L.make_cross_attention(a.pop("sequences"), a.pop("q_rows"), a.pop("kv_rows"), a.pop("heads"),
                                  a.pop("kv_heads"), a.pop("head_dim"), **a)


@pytest.mark.parametrize("kw,tiles", [
    (dict(), 2 * 2 * 2 * 2),                       # 100 queries of 2 heads: 2 blocks; 150 keys: 2
    (dict(kv_heads=4), 2 * 4 * 1 * 2), (dict(heads=6, kv_heads=2), 2 * 2 * 3 * 2),
    (dict(q_offsets=P), 2 * 2 * 4 * 2), (dict(q_offsets=P, max_q=64), 2 * 2 * 1 * 2),
    (dict(kv_offsets=P, max_kv=1), 2 * 2 * 2 * 1), (dict(kv_offsets=P, max_kv=999), 2 * 2 * 2 * 3),
    (dict(q_rows=1 << 15, kv_rows=1 << 15, heads=8, kv_heads=8, sequences=1), 256 * 256),
    (dict(head_dim=96), 0), (dict(q_rows=201), 0)])
def test_workspace(kw, tiles):
    assert L.mc_attention_backward_cross_ws_bytes(cross(**kw)) == tiles * 32768


def test_workspace_beyond_all_memory():
    """Sequences whose bounds are not known count as long as all rows are."""
    rows = dict(sequences=256, q_rows=1 << 20, kv_rows=1 << 28, heads=128, kv_heads=1)
    c = cross(q_offsets=P, kv_offsets=P, **rows)
    assert L.mc_attention_backward_cross_ws_bytes(c) == 0
    assert cross_calls(c)[1] == L.MC_ERR_UNSUPPORTED
    c = cross(q_offsets=P, kv_offsets=P, max_q=1 << 12, max_kv=1 << 20, **rows)
    assert L.mc_attention_backward_cross_ws_bytes(c) == 256 * 4096 * 8192 * 32768
    assert cross_calls(c, ws_bytes=0)[1] == L.MC_ERR_WORKSPACE


def test_norm_scratch():
    assert L.mc_qk_norm_scratch_floats(1, 2, 1, 64) == 3 * 2 * 64
    assert L.mc_qk_norm_scratch_floats(4096, 64, 64, 128) == 512 * 2 * 128
    for bad in ((0, 1, 1, 64), (4, 0, 0, 64), (4, 1, -1, 64), (4, 1, 1, 0), (4, 1, 1, 257)):
        assert L.mc_qk_norm_scratch_floats(*bad) == 0


# ------------------------------------------------------------------ refusals
def cross_calls(c, **change):
    a = dict(q=P, k=P, v=P, o=P, lse=P, dout=P, dq=P, dk=P, dv=P, delta=P, ws=P, ws_bytes=1 << 40)
    a.update(change)
    ref = None if c is None else ctypes.byref(c)
    back = [a[n] for n in ("q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv", "delta")]
    return (L.lib().mc_attention_forward_cross(*back[:5], ref, None, None),
            L.lib().mc_attention_backward_cross(*back, ref, a["ws"], a["ws_bytes"], None, None))


@pytest.mark.parametrize("kw,code", [
    (dict(sequences=0), L.MC_ERR_SHAPE), (dict(heads=0), L.MC_ERR_SHAPE),
    (dict(kv_heads=0), L.MC_ERR_SHAPE), (dict(kv_heads=3), L.MC_ERR_SHAPE),
    (dict(q_rows=0), L.MC_ERR_SHAPE), (dict(kv_rows=0), L.MC_ERR_SHAPE),
    (dict(q_rows=201), L.MC_ERR_SHAPE), (dict(kv_rows=301), L.MC_ERR_SHAPE),
    (dict(max_q=-1), L.MC_ERR_SHAPE), (dict(ld_q=255), L.MC_ERR_SHAPE),
    (dict(ld_kv=120), L.MC_ERR_SHAPE), (dict(ld_o=192), L.MC_ERR_SHAPE),
    (dict(head_dim=96), L.MC_ERR_UNSUPPORTED), (dict(heads=258, kv_heads=2), L.MC_ERR_UNSUPPORTED),
    (dict(heads=1 << 15, kv_heads=1 << 15), L.MC_ERR_UNSUPPORTED),
    (dict(ld_kv=1 << 32), L.MC_ERR_UNSUPPORTED), (dict(q_rows=1 << 29), L.MC_ERR_UNSUPPORTED),
    (dict(ld_q=260), L.MC_ERR_ALIGN), (dict(ld_kv=129), L.MC_ERR_ALIGN),
    (dict(ld_o=264), L.MC_ERR_ALIGN),    # grouped heads: rows of whole heads
    (dict(q_lens=P + 2), L.MC_ERR_ALIGN), (dict(kv_offsets=P + 1), L.MC_ERR_ALIGN),
    (dict(scale=-1.0), L.MC_ERR_ARGUMENT), (dict(scale=1e6), L.MC_ERR_ARGUMENT),
    (dict(scale=float("nan")), L.MC_ERR_ARGUMENT), (dict(scale=1e-9), L.MC_ERR_ARGUMENT),
])
def test_cross_refusals(kw, code):
    assert cross_calls(cross(**kw)) == (code, code)


def test_cross_pointer_refusals():
    assert cross_calls(None) == (L.MC_ERR_NULLPTR,) * 2
    for n in ("q", "k", "v", "o", "lse"):
        assert cross_calls(cross(), **{n: None}) == (L.MC_ERR_NULLPTR,) * 2
        assert cross_calls(cross(), **{n: P + 2}) == (L.MC_ERR_ALIGN,) * 2
    for n in ("dout", "dq", "dk", "dv", "delta", "ws"):
        assert cross_calls(cross(), **{n: None})[1] == L.MC_ERR_NULLPTR
        assert cross_calls(cross(), **{n: P + 2})[1] == L.MC_ERR_ALIGN
    need = L.mc_attention_backward_cross_ws_bytes(cross())
    assert cross_calls(cross(), ws_bytes=need - 1)[1] == L.MC_ERR_WORKSPACE


NORM = dict(x=P, dout=P, out=P, bf16=1, tokens=4, qh=2, kh=1, d=64, ld_in=192, ld_dout=192, ld_out=192,
            norm="", pos=P, freq=P, spec="", grads=None, scratch=None)


def norm_calls(**change):
    a = dict(NORM, **change)
    norm = L.make_qk_norm() if a["norm"] == "" else a["norm"]
    spec = L.make_rotary_spec(64) if a["spec"] == "" else a["spec"]
    ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
    tail = (ref(norm), a["pos"], a["freq"], ref(spec))
    heads = (a["bf16"], a["tokens"], a["qh"], a["kh"], a["d"])
    return (L.lib().mc_qk_norm_forward(a["x"], a["out"], *heads, a["ld_in"], a["ld_out"], *tail, None,
                                       None),
            L.lib().mc_qk_norm_backward(a["x"], a["dout"], a["out"], *heads, a["ld_in"], a["ld_dout"],
                                        a["ld_out"], *tail, ref(a["grads"]), 0, a["scratch"], None,
                                        None))


@pytest.mark.parametrize("change,code", [
    (dict(tokens=0), L.MC_ERR_SHAPE), (dict(qh=-1), L.MC_ERR_SHAPE), (dict(qh=0, kh=0), L.MC_ERR_SHAPE),
    (dict(d=0, spec=None), L.MC_ERR_SHAPE), (dict(ld_in=191), L.MC_ERR_SHAPE),
    (dict(ld_out=100), L.MC_ERR_SHAPE), (dict(d=62), L.MC_ERR_SHAPE),   # less than what turns
    (dict(d=257, ld_in=999, ld_out=999, ld_dout=999), L.MC_ERR_UNSUPPORTED),
    (dict(qh=1 << 17, ld_in=1 << 24, ld_out=1 << 24, ld_dout=1 << 24), L.MC_ERR_UNSUPPORTED),
    (dict(x=None), L.MC_ERR_NULLPTR), (dict(out=None), L.MC_ERR_NULLPTR),
    (dict(norm=None), L.MC_ERR_NULLPTR), (dict(pos=None), L.MC_ERR_NULLPTR),
    (dict(freq=None), L.MC_ERR_NULLPTR), (dict(x=P + 1), L.MC_ERR_ALIGN),
    (dict(bf16=0, out=P + 2), L.MC_ERR_ALIGN), (dict(pos=P + 2), L.MC_ERR_ALIGN),
    (dict(norm=L.make_qk_norm(P + 1)), L.MC_ERR_ALIGN),
    (dict(norm=L.make_qk_norm(eps=0.0)), L.MC_ERR_ARGUMENT),
    (dict(norm=L.make_qk_norm(eps=float("nan"))), L.MC_ERR_ARGUMENT),
    (dict(norm=L.make_qk_norm(eps=2.0)), L.MC_ERR_ARGUMENT),
    (dict(ld_out=256), L.MC_ERR_ARGUMENT),       # in place with another stride
])
def test_norm_refusals(change, code):
    assert norm_calls(**change) == (code, code)


def test_norm_backward_refusals():
    bad = L.make_qk_norm()
    bad.flags = 2
    assert norm_calls(norm=bad) == (L.MC_ERR_ARGUMENT,) * 2
    assert norm_calls(dout=None)[1] == L.MC_ERR_NULLPTR
    assert norm_calls(ld_dout=100, x=2 * P)[1] == L.MC_ERR_SHAPE
    assert norm_calls(ld_dout=256, x=2 * P)[1] == L.MC_ERR_ARGUMENT
    assert norm_calls(dout=P + 1)[1] == L.MC_ERR_ALIGN
    grads = L.make_qk_norm_grads(q_gain=P)
    assert norm_calls(grads=grads)[1] == L.MC_ERR_NULLPTR          # no scratch
    assert norm_calls(grads=grads, scratch=P + 2)[1] == L.MC_ERR_ALIGN
    assert norm_calls(grads=L.make_qk_norm_grads(k_shift=P + 1), scratch=P)[1] == L.MC_ERR_ALIGN


# ------------------------------------------------------------------ the binding's checks
def test_binding_refuses_arrays():
    with pytest.raises(TypeError, match="int32"):
        cross(kv_lens=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="3 elements"):
        cross(q_offsets=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="contiguous"):
        cross(q_lens=torch.zeros(2, 2, dtype=torch.int32)[:, 0])
    with pytest.raises(TypeError, match="bfloat16"):
        L.make_qk_norm(torch.ones(64))
    with pytest.raises(TypeError, match="float32"):
        L.make_qk_norm_grads(torch.ones(64, dtype=torch.bfloat16))
    c = cross()
    good = dict(q=torch.zeros(200, 256), k=torch.zeros(300, 128))
    with pytest.raises(TypeError, match="q: bfloat16"):
        L.mc_attention_forward_cross(good["q"], None, None, None, None, c)
    with pytest.raises(ValueError, match="on the GPU"):
        L.mc_attention_forward_cross(good["q"].bfloat16(), None, None, None, None, c)
    x = torch.zeros(4, 192, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="norms"):
        L.mc_qk_norm_forward(x, x.float(), 4, 2, 1, 64, 192, 192, L.make_qk_norm())
    with pytest.raises(TypeError, match="norms"):
        L.mc_qk_norm_backward(x, x.float(), x, 4, 2, 1, 64, 192, 192, 192, L.make_qk_norm())
