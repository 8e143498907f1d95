"""The layer with norms of its queries and keys, against torch in float64; and the
norms with the attention to another length, as a decoder would run them together."""
import math

import numpy as np
import pytest
import torch

import oracle.cross_attention as O
from megatron_transformer_layer_gb300 import _lib as L
from megatron_transformer_layer_gb300.layer import TransformerLayer

from gpu_util import DEV, check_status, status, to_f64
from parity import assert_close, metrics
from test_gpu_attention_opt import gen, make_documents

pytestmark = pytest.mark.gpu

B, S, HID, H, F, D = 2, 152, 256, 4, 512, 64
T = B * S
TOL = (2e-2, 2e-3)  # the layer's own gate


def vec(seed, at, d=D):
    return (at + 0.2 * torch.randn(d, generator=gen(seed))).bfloat16().to(DEV)


def make_norm(centred, shifts=True):
    return L.make_qk_norm(vec(1, 1.0), vec(2, 1.0), vec(3, 0.0) if shifts else None,
                          vec(4, 0.0) if shifts else None, eps=1e-3, centred=centred)


def torch_layer(x, w, norm, n, rot, lo, hi):
    """The layer in torch float64; n: gains and shifts (q_gain, q_shift, k_gain, k_shift)."""
    b, s, h = x.shape
    ln = lambda v, g, c: torch.nn.functional.layer_norm(v, (h,), g, c, 1e-5)  # noqa: E731
    qkv = ln(x, w["ln1_g"], w["ln1_b"]) @ w["w_qkv"].T + w["b_qkv"]
    q, k, v = (t.reshape(b, s, H, D).transpose(1, 2) for t in qkv.split(H * D, dim=-1))

    def normed(t, gain, shift):
        if norm.flags & L.MC_QK_NORM_CENTRED:
            t = t - t.mean(-1, keepdim=True)
        t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + norm.eps)
        return t * gain + (0.0 if shift is None else shift)

    q, k = normed(q, *n[:2]), normed(k, *n[2:])
    if rot is not None:
        pos, freq = rot
        ang = pos[0].double()[:, None] * freq.double()
        cos, sin = torch.cos(ang).view(b, 1, s, -1), torch.sin(ang).view(b, 1, s, -1)

        def turn(t):
            u, z = t.chunk(2, dim=-1)
            return torch.cat([u * cos - z * sin, u * sin + z * cos], -1)
        q, k = turn(q), turn(k)
    z = q @ k.transpose(-1, -2) / math.sqrt(D)
    i = torch.arange(s)
    seen = (i >= lo[:, None, :, None]) & (i < hi[:, None, :, None])
    p = torch.softmax(z.masked_fill(~seen, -1e300), -1) * seen
    o = (p @ v).transpose(1, 2).reshape(b, s, -1)
    x1 = x + o @ w["w_o"].T + w["b_o"]
    u = ln(x1, w["ln2_g"], w["ln2_b"]) @ w["w_fc1"].T + w["b_fc1"]
    return x1 + torch.nn.functional.gelu(u, approximate="tanh") @ w["w_fc2"].T + w["b_fc2"]


NAMES = ("q_norm_g", "q_norm_b", "k_norm_g", "k_norm_b")


@pytest.mark.parametrize("flags", [dict(), dict(recompute=True), dict(sequence_parallel=True),
                                   dict(fp8=True), dict(accumulate_grads=True)])
@pytest.mark.parametrize("centred,rotary,mask", [(True, True, True), (False, True, False),
                                                 (False, False, False)])
def test_layer_with_norms(flags, centred, rotary, mask):
    params = TransformerLayer.random_params(HID, H, F, seed=3, std=0.05)
    params["b_qkv"] = (0.1 * torch.randn(3 * H * D, generator=gen(9))).bfloat16().to(DEV)
    pos = torch.randint(0, 400, (1, T), generator=gen(11), dtype=torch.int32)
    freq = torch.rand(32, generator=gen(12))
    rot = L.make_layer_rotary(L.make_rotary_spec(64), pos.to(DEV), freq.to(DEV)) if rotary else None
    lo, hi = torch.zeros(B, S, dtype=torch.int64), torch.arange(1, S + 1).expand(B, S)
    att = None
    if mask:
        klo, khi, tab = make_documents([0, 40, 152, 250, 300], None, True, 0, B, S)
        lo, hi = klo.cpu().long(), khi.cpu().long()
        att = L.make_attention_options(klo, khi, tab)
    norm = make_norm(centred, shifts=centred)
    layer = TransformerLayer(B, S, HID, H, F, 2, params=params, rotary=rot, attention=att,
                             qk_norm=norm, **flags)
    x, dy = (torch.randn(T, HID, generator=gen(k)).to(DEV) for k in (1, 2))
    passes = 2 if flags.get("accumulate_grads") else 1
    for _ in range(passes):
        y, dx = layer.forward(x), layer.backward(dy)
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    assert [n for n in NAMES if n in layer.grads] == [n for n, t in zip(NAMES, norm.tensors)
                                                      if t is not None]
    w = {n: v.detach().double().cpu().requires_grad_() for n, v in params.items()}
    n64 = [None if t is None else t.double().cpu().requires_grad_() for t in norm.tensors]
    x64 = x.double().cpu().view(B, S, HID).requires_grad_()
    y64 = torch_layer(x64, w, norm, n64, (pos, freq) if rotary else None, lo, hi)
    y64.backward(dy.double().cpu().view(B, S, HID))
    # 8-bit operands: 2^-2 of a tensor's size for the largest error and 2^-4 on
    # average, counted in the test of positions and masks
    tol = TOL if not flags.get("fp8") else (2.0 ** -2, 2.0 ** -4)
    assert_close("y", to_f64(y), y64.detach().numpy().reshape(T, HID), *tol)
    assert_close("dx", to_f64(dx), x64.grad.numpy().reshape(T, HID), *tol)
    for n in w:
        assert_close(n, to_f64(layer.grads[n]), passes * w[n].grad.numpy(), *tol)
    # The norms' gradients are sums over tokens and heads of values of either sign,
    # each off by the roundings on its way: of LN1's output, Q, K and V, the normed
    # Q and K, P, the three gradients before dO, dO, delta's O, dz and dQ or dK, at
    # least ten, each at most half a step, 2^-8 of the value, and of either sign. A
    # sum's error is to its size as a value's is to its own: at most sqrt(10) 2^-8
    # in the mean of 64 sums.
    for n, t in zip(NAMES, n64):
        if t is not None:
            m = metrics(to_f64(layer.grads[n]), passes * t.grad.numpy())
            mean = math.sqrt(10) * 2.0 ** -8 if not flags.get("fp8") else tol[0]
            assert m["finite"] and m["max_rel"] <= tol[0] and m["norm_rel"] <= mean, (n, m)


@pytest.mark.parametrize("gains", [True, False])
def test_heads_of_128(gains):
    """Heads of 128: the layer against its parts, the norms and the attention by their
    stage calls and the rest in float64."""
    heads, d = 2, 128
    a = heads * d
    params = TransformerLayer.random_params(HID, heads, F, seed=3, std=0.05)
    norm = L.make_qk_norm(*((vec(1, 1.0, d), vec(2, 1.0, d)) if gains else ()), eps=1e-3)
    layer = TransformerLayer(B, S, HID, heads, F, params=params, qk_norm=norm)
    x, dy = (torch.randn(T, HID, generator=gen(k)).to(DEV) for k in (1, 2))
    y, dx = layer.forward(x), layer.backward(dy)
    assert layer.device_status() == 0
    o, st = torch.empty(T, a, dtype=torch.bfloat16, device=DEV), status()
    lse = torch.empty(B * heads * S, device=DEV)
    ln1 = torch.nn.functional.layer_norm(x.double(), (HID,), params["ln1_g"].double(),
                                         params["ln1_b"].double(), 1e-5)
    qkv = (ln1.bfloat16().double() @ params["w_qkv"].double().T + params["b_qkv"].double()).bfloat16()
    assert L.mc_qk_norm_forward(qkv, qkv, T, heads, heads, d, 3 * a, 3 * a, norm, status=st) == 0
    assert L.mc_attention_forward(qkv, o, lse, B, S, heads, d, st, torch.cuda.current_stream()) == 0
    check_status(st)
    x1 = x.double() + o.double() @ params["w_o"].double().T + params["b_o"].double()
    ln2 = torch.nn.functional.layer_norm(x1, (HID,), params["ln2_g"].double(),
                                         params["ln2_b"].double(), 1e-5)
    u = ln2 @ params["w_fc1"].double().T + params["b_fc1"].double()
    want = x1 + torch.nn.functional.gelu(u, approximate="tanh") @ params["w_fc2"].double().T + \
        params["b_fc2"].double()
    assert_close("y", to_f64(y), want.cpu().numpy(), *TOL)
    assert [n for n in NAMES if n in layer.grads] == (["q_norm_g", "k_norm_g"] if gains else [])
    assert bool(torch.isfinite(dx).all())


def test_layer_without_norms_keeps_its_bits():
    params = TransformerLayer.random_params(HID, H, F, seed=3, std=0.05)
    layer = TransformerLayer(B, S, HID, H, F, 2, params=params)
    x, dy = (torch.randn(T, HID, generator=gen(k)).to(DEV) for k in (1, 2))
    y, dx = layer.forward(x), layer.backward(dy)
    want = [t.clone() for t in (y, dx, *layer.grads.values())]
    y2, dx2 = torch.empty_like(y), torch.empty_like(dx)
    assert L.mc_layer_forward(layer.shape, layer.weights, x, y2, layer.saved, layer.ws,
                              layer.ws_bytes, torch.cuda.current_stream()) == 0
    assert L.mc_layer_backward(layer.shape, layer.weights, x, dy, layer.saved, dx2, layer._grads_c,
                               layer.ws, layer.ws_bytes, torch.cuda.current_stream()) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (y2, dx2, *layer.grads.values())))


def test_other_norms_and_a_graph():
    """Norms changed from step to step; a captured step gives an eager one's bits."""
    params = TransformerLayer.random_params(HID, H, F, seed=3, std=0.05)
    a, b = make_norm(True), make_norm(False)
    layer = TransformerLayer(B, S, HID, H, F, params=params, qk_norm=a)
    x, dy = (torch.randn(T, HID, generator=gen(k)).to(DEV) for k in (1, 2))

    def step():
        y, dx = layer.forward(x), layer.backward(dy)
        torch.cuda.synchronize()
        return [t.clone() for t in (y, dx, *layer.grads.values())]

    first = step()
    layer.set_qk_norm(b)
    other = step()
    assert not torch.equal(first[0], other[0])
    layer.set_qk_norm(a)
    assert all(torch.equal(u, v) for u, v in zip(step(), first))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer.forward(x, y)
        layer.backward(dy, dx)
    for t in layer.grads.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip((y, dx, *layer.grads.values()), first))
    with pytest.raises(ValueError, match="without norms"):
        TransformerLayer(B, S, HID, H, F, params=params).set_qk_norm(a)


def test_norms_that_do_not_cover_a_head():
    params = TransformerLayer.random_params(HID, H, F, seed=3)
    layer = TransformerLayer(B, S, HID, H, F, params=params, qk_norm=make_norm(True))
    x = torch.randn(T, HID, generator=gen(1)).to(DEV)
    with pytest.raises(ValueError, match="with norms"):
        layer.set_qk_norm(None)
    short = L.make_qk_norm(vec(1, 1.0), vec(2, 1.0, D - 1))
    layer.set_qk_norm(short)
    with pytest.raises(ValueError, match="norm of k: 64 elements"):
        layer.forward(x)
    w = (layer.shape, layer.weights, L.make_layer_qk_norm(
        make_norm(True), L.make_qk_norm_grads(torch.zeros(32, device=DEV))), None, None)
    with pytest.raises(ValueError, match="gradient of q: 64 elements"):
        L.mc_layer_backward_norm(*w, x, x, layer.saved, x, layer._grads_c, layer.ws, layer.ws_bytes)


@pytest.mark.parametrize("heads,kv_heads,d", [(4, 4, 64), (6, 2, 128)])
def test_a_decoders_cross_attention(heads, kv_heads, d):
    """Queries from one tensor, keys from another, each normed (the keys turned
    too), attention between them, and all of it back, against the float64 parts."""
    n, sq, sk = 3, 70, 190
    a, akv = heads * d, kv_heads * d
    bf16 = lambda k, *s: torch.randn(*s, generator=gen(k)).bfloat16().to(DEV)  # noqa: E731
    q, kv, dout = bf16(1, n * sq, a), bf16(2, n * sk, 2 * akv), bf16(3, n * sq, a)
    lens = [190, 0, 77]
    norm = L.make_qk_norm(vec(1, 1.0, d), vec(2, 1.0, d), eps=1e-5)
    pos = torch.randint(0, 3000, (1, n * sk), generator=gen(5), dtype=torch.int32).to(DEV)
    freq = torch.rand(d // 2, generator=gen(6)).to(DEV)
    spec = L.make_rotary_spec(d)
    st = status()
    qn, kn = torch.empty_like(q), torch.empty(n * sk, akv, dtype=torch.bfloat16, device=DEV)
    o, lse = torch.empty_like(q), torch.empty(heads, n * sq, device=DEV)
    c = L.make_cross_attention(n, n * sq, n * sk, heads, kv_heads, d, ld_kv=2 * akv,
                               kv_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    # the normed keys beside the values they belong to
    kvn = kv.clone()
    assert L.mc_qk_norm_forward(q, qn, n * sq, heads, 0, d, a, a, norm, status=st) == 0
    assert L.mc_qk_norm_forward(kv, kvn, n * sk, 0, kv_heads, d, 2 * akv, 2 * akv, norm, pos, freq,
                                spec, st) == 0
    assert torch.equal(kvn[:, akv:], kv[:, akv:])
    kn, v = kvn[:, :akv], kvn[:, akv:]
    assert L.mc_attention_forward_cross(qn, kn, v, o, lse, c, st) == 0
    dqn, dkv = torch.empty_like(q), torch.empty_like(kv)
    delta = torch.empty_like(lse)
    ws_bytes = L.mc_attention_backward_cross_ws_bytes(c)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=DEV)
    assert L.mc_attention_backward_cross(qn, kn, v, o, lse, dout, dqn, dkv[:, :akv], dkv[:, akv:],
                                         delta, c, ws, ws_bytes, st) == 0
    got_qn, got_kn, got_dqn, got_dkv = (to_f64(t) for t in (qn, kn, dqn, dkv))
    grads = torch.empty(2, d, device=DEV)
    scratch = torch.empty(L.mc_qk_norm_scratch_floats(n * sk, heads, kv_heads, d), device=DEV)
    # the gradients go on in place
    assert L.mc_qk_norm_backward(q, dqn, dqn, n * sq, heads, 0, d, a, a, a, norm,
                                 grads=L.make_qk_norm_grads(q_gain=grads[0]), scratch=scratch,
                                 status=st) == 0
    assert L.mc_qk_norm_backward(kv, dkv, dkv, n * sk, 0, kv_heads, d, 2 * akv, 2 * akv, 2 * akv, norm,
                                 pos, freq, spec, L.make_qk_norm_grads(k_gain=grads[1]), 0, scratch,
                                 st) == 0
    check_status(st)
    # each part against its oracle, on the bf16 values it got
    turn = (pos.cpu().numpy(), freq.cpu().numpy(), d, [d // 2])
    g = [to_f64(t) for t in (norm.tensors[0], norm.tensors[2])]
    q64, kv64 = to_f64(q), to_f64(kv)
    want = O.qk_norm(q64.reshape(-1, heads, d), heads, 0, 1e-5, False, g).reshape(-1, a)
    assert (np.abs(got_qn - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * 8).all()
    want = O.qk_norm(kv64[:, :akv].reshape(-1, kv_heads, d), 0, kv_heads, 1e-5, False, g,
                     turn=turn).reshape(-1, akv)
    assert (np.abs(got_kn - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * 8).all()
    seqs = O.sequence_rows(n, n * sq), O.sequence_rows(n, n * sk, None, lens)
    args = (*seqs, heads, kv_heads, d, 1.0 / math.sqrt(d))
    ref, _, tol, _, _ = O.forward(got_qn, got_kn, kv64[:, akv:], *args)
    assert (np.abs(to_f64(o) - ref) <= tol).all()
    (dq_, dk_, dv_), tols, _ = O.backward(got_qn, got_kn, kv64[:, akv:], to_f64(dout), *args)
    assert (np.abs(got_dqn - dq_) <= tols[0]).all()
    assert (np.abs(got_dkv - np.concatenate([dk_, dv_], 1)) <= np.concatenate(tols[1:], 1)).all()
    dx, size, sums = O.qk_norm_backward(q64.reshape(-1, heads, d), got_dqn.reshape(-1, heads, d), heads,
                                        0, 1e-5, False, g)
    tol = 2.0 ** -8 * np.abs(dx) + 2.0 ** -18 * size.max(axis=2, keepdims=True)
    assert (np.abs(to_f64(dqn).reshape(dx.shape) - dx) <= tol).all()
    assert np.abs(to_f64(grads[0]) - sums[0][0][0]).max() <= 2.0 ** -18 * sums[0][0][1].max()
    dx, size, sums = O.qk_norm_backward(kv64[:, :akv].reshape(-1, kv_heads, d),
                                        got_dkv[:, :akv].reshape(-1, kv_heads, d), 0, kv_heads, 1e-5,
                                        False, g, turn)
    tol = 2.0 ** -8 * np.abs(dx) + 2.0 ** -18 * size.max(axis=2, keepdims=True)
    assert (np.abs(to_f64(dkv[:, :akv]).reshape(dx.shape) - dx) <= tol).all()
    assert np.array_equal(to_f64(dkv[:, akv:]), got_dkv[:, akv:])
    assert np.abs(to_f64(grads[1]) - sums[0][1][0]).max() <= 2.0 ** -18 * sums[0][1][1].max()
