"""Rotary positions, interval masks and attention over them, without a GPU:
the float64 oracle against plainer forms and differences, workspace sizes, and
what the entry points refuse before anything is launched."""
import ctypes
import math

import numpy as np
import pytest

import oracle.attention_opt as O
from megatron_transformer_layer_gb300 import _lib as L

P = 1 << 20  # a pointer that is aligned and never dereferenced


# ------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("adjacent", [False, True])
def test_rotary_oracle_is_a_rotation(adjacent):
    g = np.random.default_rng(1)
    x = g.standard_normal((5, 2, 16))
    pos = g.integers(-50, 50, (2, 5))
    f = (10000.0 ** (-np.arange(6) / 6)).astype(np.float32)
    a = dict(rot_dim=12, sections=[4, 2], adjacent=adjacent)
    y = O.rotary(x, pos, f, **a)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-13)
    assert np.array_equal(y[:, :, 12:], x[:, :, 12:])
    assert np.allclose(O.rotary(y, pos, f, inverse=True, **a), x, atol=1e-13)
    # a score of two rotated vectors depends on the difference of their positions alone
    q, k = g.standard_normal((1, 1, 16)), g.standard_normal((1, 1, 16))
    one = lambda v, t: O.rotary(v, np.full((2, 1), t), f, **a)[0, 0]  # noqa: E731
    assert np.isclose(one(q, 7) @ one(k, 3), one(q, 1004) @ one(k, 1000), atol=1e-12)


def test_rotary_oracle_far_positions():
    # 10^6 turns of an angle of 1: against numpy's own argument reduction in float64
    for t in (1, 10 ** 6, 2 ** 31 - 1, -(2 ** 31)):
        assert math.isclose(math.cos(O._reduced(t, 1.0)), math.cos(float(t)), abs_tol=1e-6)
        assert math.isclose(math.sin(O._reduced(t, 1.0)), math.sin(float(t)), abs_tol=1e-6)


def test_axes_dealt_in_turn():
    assert O.axis_of_pair([3, 1, 2], dealt=True) == [0, 1, 2, 0, 2, 0]
    assert O.axis_of_pair([3, 1, 2]) == [0, 0, 0, 1, 2, 2]


@pytest.mark.parametrize("cap,bias", [(0.0, False), (3.0, False), (0.0, True), (3.0, True)])
def test_attention_oracle_against_differences(cap, bias):
    """The backward formula against central differences of the forward."""
    g = np.random.default_rng(2)
    b, s, H, d = 1, 9, 2, 4
    qkv = g.standard_normal((b, s, 3 * H * d)) * 1.5
    dout = g.standard_normal((b, s, H * d))
    lo = np.array([[0, 0, 0, 3, 3, 3, 3, 0, 6]])
    hi = np.array([[1, 2, 5, 4, 5, 9, 7, 0, 9]])   # token 7 sees nothing
    slopes = np.array([0.5, 0.0625]) if bias else None
    f = lambda x: (O.attention_forward(x, lo, hi, H, d, slopes, cap)[0] * dout).sum()  # noqa: E731
    got = O.attention_backward(qkv, dout, lo, hi, H, d, slopes, cap)[0]
    eps = 1e-5
    for at in np.ndindex(qkv.shape):
        x = qkv.copy()
        x[at] += eps
        up = f(x)
        x[at] -= 2 * eps
        assert abs((up - f(x)) / (2 * eps) - got[at]) < 1e-8
    o, lse, _, _ = O.attention_forward(qkv, lo, hi, H, d, slopes, cap)
    assert (o[0, 7] == 0).all() and (lse[0, :, 7] == -np.inf).all()


def test_document_intervals_oracle():
    lo, hi = O.document_intervals([0, 3, 3, 8, 10], [2, 0, 4, -1], True, 0, 2, 6)
    # document 2 runs over the end of the first sequence and is cut there
    assert lo.tolist() == [[0, 0, 0, 3, 3, 3], [0, 0, 0, 0, 0, 0]]
    assert hi.tolist() == [[2, 2, 3, 6, 6, 6], [1, 2, 0, 0, 0, 0]]


# ------------------------------------------------------------------ sizes
@pytest.mark.parametrize("b,s,ints", [(1, 1, 8), (1, 128, 8), (1, 129, 16), (3, 300, 72),
                                      (0, 4, 0), (1, 0, 0), (1 << 12, 1 << 13, 0)])
def test_mask_table_ints(b, s, ints):
    assert L.mc_attention_mask_table_ints(b, s) == ints


@pytest.mark.parametrize("b,s,H,d,causal,tiles", [
    (1, 128, 2, 64, True, 2), (1, 129, 2, 64, True, 6), (2, 400, 3, 128, False, 96),
    (1, 128, 2, 96, True, 0), (1, 0, 2, 64, True, 0)])
def test_backward_workspace(b, s, H, d, causal, tiles):
    opt = L.make_attention_options(None, None, None, causal=causal)
    assert L.mc_attention_backward_opt_ws_bytes(b, s, H, d, opt) == tiles * 32768


def test_layer_workspace_covers_the_tiles():
    sh = L.make_shape(1, 500, 768, 12, 2304)
    causal = L.make_attention_options(P, P, P)
    ahead = L.make_attention_options(P, P, P, causal=False)
    base = L.mc_layer_workspace_bytes(sh)
    assert L.mc_layer_workspace_bytes_opt(sh, None) == base
    assert L.mc_layer_workspace_bytes_opt(sh, causal) == base
    assert L.mc_layer_workspace_bytes_opt(sh, ahead) == base + 12 * 6 * 32768  # 16 tiles, not 10


# ------------------------------------------------------------------ refusals
def spec(rot=64, sections=None, **kw):
    return L.make_rotary_spec(rot, sections, **kw)


ROTARY = dict(x=P, out=P, bf16=1, tokens=4, heads=2, d=64, ld_in=128, ld_out=128, pos=P, freq=P,
              spec=None)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=0), L.MC_ERR_SHAPE), (dict(heads=0), L.MC_ERR_SHAPE), (dict(d=0), L.MC_ERR_SHAPE),
    (dict(ld_in=127), L.MC_ERR_SHAPE), (dict(ld_out=64), L.MC_ERR_SHAPE),
    (dict(spec=spec(66)), L.MC_ERR_SHAPE), (dict(spec=spec(31, [15])), L.MC_ERR_SHAPE),
    (dict(spec=spec(0, [0])), L.MC_ERR_SHAPE), (dict(spec=spec(64, [16, 15])), L.MC_ERR_SHAPE),
    (dict(spec=spec(64, [40, -8])), L.MC_ERR_SHAPE),
    (dict(x=None), L.MC_ERR_NULLPTR), (dict(out=None), L.MC_ERR_NULLPTR),
    (dict(pos=None), L.MC_ERR_NULLPTR), (dict(freq=None), L.MC_ERR_NULLPTR),
    (dict(x=P + 1), L.MC_ERR_ALIGN), (dict(bf16=0, out=P + 2), L.MC_ERR_ALIGN),
    (dict(pos=P + 2), L.MC_ERR_ALIGN),
    (dict(ld_out=160), L.MC_ERR_ARGUMENT),       # in place with another stride
    (dict(d=1024, ld_in=4096, ld_out=4096, spec=spec(514)), L.MC_ERR_UNSUPPORTED),
    (dict(d=1026, ld_in=4096, ld_out=4096), L.MC_ERR_UNSUPPORTED),
    (dict(heads=1, d=3000000, ld_in=1 << 22, ld_out=1 << 22), L.MC_ERR_UNSUPPORTED),
    (dict(heads=65537, ld_in=1 << 23, ld_out=1 << 23), L.MC_ERR_UNSUPPORTED),
])
def test_rotary_refusals(change, code):
    a = dict(ROTARY, spec=spec())
    a.update(change)
    for fn in (L.lib().mc_rotary_forward, L.lib().mc_rotary_backward):
        assert fn(a["x"], a["out"], a["bf16"], a["tokens"], a["heads"], a["d"], a["ld_in"],
                  a["ld_out"], a["pos"], a["freq"], ctypes.byref(a["spec"]), None, None) == code


def test_rotary_spec_refusals():
    bad = spec()
    bad.axes = 5
    assert L.lib().mc_rotary_forward(P, P, 1, 4, 2, 64, 128, 128, P, P, ctypes.byref(bad), None,
                                     None) == L.MC_ERR_ARGUMENT
    bad = spec()
    bad.flags = 8
    assert L.lib().mc_rotary_forward(P, P, 1, 4, 2, 64, 128, 128, P, P, ctypes.byref(bad), None,
                                     None) == L.MC_ERR_ARGUMENT
    assert L.lib().mc_rotary_forward(P, P, 1, 4, 2, 64, 128, 128, P, P, None, None,
                                     None) == L.MC_ERR_NULLPTR
    with pytest.raises(ValueError):
        L.make_rotary_spec(64, [8] * 5)
    with pytest.raises(ValueError):
        L.make_rotary_spec(64, [])


DOCS = dict(off=P, n=3, pre=P, causal=1, window=0, b=2, s=100, lo=P, hi=P, tab=P)


@pytest.mark.parametrize("change,code", [
    (dict(b=0), L.MC_ERR_SHAPE), (dict(s=-1), L.MC_ERR_SHAPE),
    (dict(b=1 << 10, s=1 << 20), L.MC_ERR_UNSUPPORTED), (dict(b=70000, s=1), L.MC_ERR_UNSUPPORTED),
    (dict(n=-1), L.MC_ERR_ARGUMENT), (dict(window=-1), L.MC_ERR_ARGUMENT),
    (dict(off=None), L.MC_ERR_NULLPTR), (dict(lo=None), L.MC_ERR_NULLPTR),
    (dict(hi=None), L.MC_ERR_NULLPTR), (dict(tab=None), L.MC_ERR_NULLPTR),
    (dict(off=P + 2), L.MC_ERR_ALIGN), (dict(tab=P + 4), L.MC_ERR_ALIGN),
    (dict(pre=P + 1), L.MC_ERR_ALIGN),
])
def test_mask_refusals(change, code):
    a = dict(DOCS)
    a.update(change)
    assert L.mc_attention_mask_documents(a["off"], a["n"], a["pre"], a["causal"], a["window"],
                                         a["b"], a["s"], a["lo"], a["hi"], a["tab"]) == code
    if "off" not in change and "pre" not in change and "n" not in change and "window" not in change:
        assert L.mc_attention_mask_intervals(a["b"], a["s"], a["lo"], a["hi"], a["tab"]) == code


ATT = dict(qkv=P, o=P, lse=P, dout=P, dqkv=P, delta=P, b=1, s=200, H=2, d=64, lo=P, hi=P, tab=P,
           slopes=None, cap=0.0, ws=None, ws_bytes=0)


@pytest.mark.parametrize("change,code", [
    (dict(b=0), L.MC_ERR_SHAPE), (dict(s=0), L.MC_ERR_SHAPE), (dict(H=-2), L.MC_ERR_SHAPE),
    (dict(d=96), L.MC_ERR_UNSUPPORTED), (dict(H=70000), L.MC_ERR_UNSUPPORTED),
    (dict(b=1 << 12, s=1 << 13), L.MC_ERR_UNSUPPORTED),
    (dict(qkv=None), L.MC_ERR_NULLPTR), (dict(o=None), L.MC_ERR_NULLPTR),
    (dict(lse=None), L.MC_ERR_NULLPTR), (dict(lo=None), L.MC_ERR_NULLPTR),
    (dict(hi=None), L.MC_ERR_NULLPTR), (dict(tab=None), L.MC_ERR_NULLPTR),
    (dict(qkv=P + 8), L.MC_ERR_ALIGN), (dict(tab=P + 8), L.MC_ERR_ALIGN),
    (dict(slopes=P + 2), L.MC_ERR_ALIGN), (dict(lse=P + 2), L.MC_ERR_ALIGN),
    (dict(cap=-1.0), L.MC_ERR_ARGUMENT), (dict(cap=math.inf), L.MC_ERR_ARGUMENT),
    (dict(cap=math.nan), L.MC_ERR_ARGUMENT),
])
def test_attention_refusals(change, code):
    a = dict(ATT)
    a.update(change)
    opt = L.make_attention_options(a["lo"], a["hi"], a["tab"], a["slopes"], a["cap"])
    assert L.mc_attention_forward_opt(a["qkv"], a["o"], a["lse"], a["b"], a["s"], a["H"], a["d"],
                                      opt) == code
    assert L.mc_attention_backward_opt(a["qkv"], a["o"], a["lse"], a["dout"], a["dqkv"],
                                       a["delta"], a["b"], a["s"], a["H"], a["d"], opt) == code


@pytest.mark.parametrize("change,code", [
    (dict(dout=None), L.MC_ERR_NULLPTR), (dict(dqkv=None), L.MC_ERR_NULLPTR),
    (dict(delta=None), L.MC_ERR_NULLPTR), (dict(dqkv=P + 4), L.MC_ERR_ALIGN),
    (dict(ws=P, ws_bytes=3 * 2 * 32768 - 1), L.MC_ERR_WORKSPACE),
    (dict(ws=P + 8, ws_bytes=1 << 30), L.MC_ERR_ALIGN),
])
def test_attention_backward_refusals(change, code):
    a = dict(ATT)
    a.update(change)
    opt = L.make_attention_options(a["lo"], a["hi"], a["tab"])
    assert L.mc_attention_backward_opt(a["qkv"], a["o"], a["lse"], a["dout"], a["dqkv"],
                                       a["delta"], a["b"], a["s"], a["H"], a["d"], opt, a["ws"],
                                       a["ws_bytes"]) == code


@pytest.mark.parametrize("cap,code", [
    (-1.0, L.MC_ERR_ARGUMENT), (float("nan"), L.MC_ERR_ARGUMENT),
    (float("inf"), L.MC_ERR_ARGUMENT), (1e5, L.MC_ERR_ARGUMENT), (1e-6, L.MC_ERR_ARGUMENT),
    (2.0 ** 16, L.MC_ERR_NULLPTR), (2.0 ** -16, L.MC_ERR_NULLPTR), (0.0, L.MC_ERR_NULLPTR)])
def test_softcap_range(cap, code):
    """Caps in range get as far as the check of the other pointers."""
    opt = L.make_attention_options(P, P, P, softcap=cap)
    assert L.mc_attention_forward_opt(None, P, P, 1, 4, 2, 64, opt) == code
    assert L.mc_attention_backward_opt(None, P, P, P, P, P, 1, 4, 2, 64, opt) == code


def test_null_options():
    assert L.mc_attention_forward_opt(P, P, P, 1, 4, 2, 64, None) == L.MC_ERR_NULLPTR
    assert L.mc_attention_backward_opt(P, P, P, P, P, P, 1, 4, 2, 64, None) == L.MC_ERR_NULLPTR
    assert L.mc_attention_backward_opt_ws_bytes(1, 4, 2, 64, None) == 0


@pytest.mark.parametrize("rot,opt,code", [
    (dict(rot_dim=130), None, L.MC_ERR_SHAPE), (dict(positions=None), None, L.MC_ERR_NULLPTR),
    (dict(inv_freq=None), None, L.MC_ERR_NULLPTR), (dict(inv_freq=P + 2), None, L.MC_ERR_ALIGN),
    (None, dict(softcap=-2.0), L.MC_ERR_ARGUMENT), (None, dict(tables=None), L.MC_ERR_NULLPTR),
])
def test_layer_refusals(rot, opt, code):
    sh = L.make_shape(1, 64, 768, 12, 2304)
    w = L.mc_layer_weights(*[P] * 12)
    g = L.mc_layer_grads(*[P] * 12)
    r = o = None
    if rot is not None:
        a = dict(rot_dim=64, positions=P, inv_freq=P)
        a.update(rot)
        r = L.make_layer_rotary(L.make_rotary_spec(a["rot_dim"]), a["positions"], a["inv_freq"])
    if opt is not None:
        a = dict(key_lo=P, key_hi=P, tables=P, softcap=0.0)
        a.update(opt)
        o = L.make_attention_options(a["key_lo"], a["key_hi"], a["tables"], softcap=a["softcap"])
    n = L.mc_layer_workspace_bytes_opt(sh, o)
    assert L.mc_layer_forward_opt(sh, w, r, o, P, P, P, P, n) == code
    assert L.mc_layer_backward_opt(sh, w, r, o, P, P, P, P, g, P, n) == code


def test_layer_workspace_too_small_for_a_mask_that_looks_ahead():
    sh = L.make_shape(1, 500, 768, 12, 2304)
    ahead = L.make_attention_options(P, P, P, causal=False)
    n = L.mc_layer_workspace_bytes(sh)
    assert L.mc_layer_forward_opt(sh, L.mc_layer_weights(*[P] * 12), None, ahead, P, P, P, P,
                                  n) == L.MC_ERR_WORKSPACE
