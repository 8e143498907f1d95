"""The layer against its parts, to the bit: the stage calls of the library, one after
another on tensors of the test's own; with and without norms of queries and keys,
heads of 64 and 128.  And with heads of 128 against torch in float64."""
import math

import pytest
import torch

import test_gpu_layer_qk_norm as N
from megatron_transformer_layer_gb300 import _lib as L
from megatron_transformer_layer_gb300.layer import TransformerLayer

from gpu_util import DEV, check_status, status, to_f64
from parity import assert_close, metrics
from test_gpu_attention_opt import gen

pytestmark = pytest.mark.gpu

B, S, HID, F = 2, 152, 256, 512
T = B * S


def inputs(heads, d):
    params = TransformerLayer.random_params(HID, heads, F, head_dim=d, seed=3, std=0.05)
    for k, name in enumerate(("b_qkv", "b_o", "b_fc1", "b_fc2", "ln1_b", "ln2_b")):
        params[name] = (0.1 * torch.randn(params[name].shape, generator=gen(9 + k))).bfloat16().to(DEV)
    return params, *(torch.randn(T, HID, generator=gen(k)).to(DEV) for k in (1, 2))


def make_norm(kind, d):
    return {"none": lambda: None, "plain": lambda: L.make_qk_norm(eps=1e-3),
            "gains": lambda: L.make_qk_norm(N.vec(1, 1.0, d), N.vec(2, 1.0, d), eps=1e-3),
            "centred": lambda: L.make_qk_norm(N.vec(1, 1.0, d), N.vec(2, 1.0, d), N.vec(3, 0.0, d),
                                              N.vec(4, 0.0, d), eps=1e-3, centred=True)}[kind]()


class Parts:
    def __init__(self, params, heads, d, norm):
        self.w, self.heads, self.d, self.a, self.norm = params, heads, d, heads * d, norm
        self.st = status()

    def new(self, *shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=DEV)

    def f32(self, *shape):
        return self.new(*shape, dtype=torch.float32)

    def run(self, rc):
        assert rc == 0

    def gemm(self, m, n, k, x, x_layout, y, y_layout, out, epilogue, bias=None, aux=None):
        self.run(L.mc_gemm(m, n, k, x, x.stride(0), x_layout, y, y.stride(0), y_layout, out,
                           out.stride(0), epilogue, bias, aux, 0 if aux is None else aux.stride(0), 0, 1,
                           self.st, torch.cuda.current_stream()))
        return out

    def norm_rows(self, x, name):
        out, mean, rstd = self.new(T, HID), self.f32(T), self.f32(T)
        self.run(L.mc_layernorm_forward(x, self.w[name + "_g"], self.w[name + "_b"], out, mean, rstd, T,
                                        HID, self.st, torch.cuda.current_stream()))
        return out, mean, rstd

    def norm_rows_back(self, name, dout, x, stats, resid, bf16, colsum):
        dx, partials = self.f32(T, HID), self.f32(L.mc_layernorm_backward_scratch_floats(T, HID))
        g, b = self.f32(HID), self.f32(HID)
        self.run(L.mc_layernorm_backward(dout, x, *stats, self.w[name + "_g"], resid, dx, bf16, g, b,
                                         colsum, 0, partials, T, HID, self.st,
                                         torch.cuda.current_stream()))
        self.g[name + "_g"], self.g[name + "_b"] = g, b
        return dx

    def forward(self, x):
        w, a = self.w, self.a
        self.x = x
        self.ln1, *self.s1 = self.norm_rows(x, "ln1")
        self.qkv = self.new(T, 3 * a)
        if self.norm is None:
            self.gemm(T, 3 * a, HID, self.ln1, 0, w["w_qkv"], 0, self.qkv, 2, w["b_qkv"])
        else:
            self.raw = self.gemm(T, 2 * a, HID, self.ln1, 0, w["w_qkv"], 0, self.new(T, 2 * a), 2,
                                 w["b_qkv"])
            self.gemm(T, a, HID, self.ln1, 0, w["w_qkv"][2 * a:], 0, self.qkv[:, 2 * a:], 2,
                      w["b_qkv"][2 * a:])
            self.run(L.mc_qk_norm_forward(self.raw, self.qkv, T, self.heads, self.heads, self.d, 2 * a,
                                          3 * a, self.norm, status=self.st))
        self.o, self.lse = self.new(T, a), self.f32(self.heads * T)
        self.run(L.mc_attention_forward(self.qkv, self.o, self.lse, B, S, self.heads, self.d, self.st,
                                        torch.cuda.current_stream()))
        self.x1 = self.gemm(T, HID, a, self.o, 0, w["w_o"], 0, self.f32(T, HID), 4, w["b_o"], x)
        self.ln2, *self.s2 = self.norm_rows(self.x1, "ln2")
        self.hp = self.new(T, F)
        self.act = self.gemm(T, F, HID, self.ln2, 0, w["w_fc1"], 0, self.new(T, F), 3, w["b_fc1"], self.hp)
        return self.gemm(T, HID, F, self.act, 0, w["w_fc2"], 0, self.f32(T, HID), 4, w["b_fc2"], self.x1)

    def backward(self, dy):
        """dx, the gradients that are formed by stage calls, and the rows whose column
        sums are the others."""
        w, a, g = self.w, self.a, {}
        self.g = g
        dy16 = dy.bfloat16()
        g["w_fc2"] = self.gemm(HID, F, T, dy16, 1, self.act, 1, self.f32(HID, F), 0)
        dhp = self.gemm(T, F, HID, dy16, 0, w["w_fc2"], 1, self.new(T, F), 5, aux=self.hp)
        g["w_fc1"] = self.gemm(F, HID, T, dhp, 1, self.ln2, 1, self.f32(F, HID), 0)
        dln = self.gemm(T, HID, F, dhp, 0, w["w_fc1"], 1, self.f32(T, HID), 0)
        dx1_16, g["b_o"] = self.new(T, HID), self.f32(HID)
        dx1 = self.norm_rows_back("ln2", dln, self.x1, self.s2, dy, dx1_16, g["b_o"])
        g["w_o"] = self.gemm(HID, a, T, dx1_16, 1, self.o, 1, self.f32(HID, a), 0)
        do = self.gemm(T, a, HID, dx1_16, 0, w["w_o"], 1, self.new(T, a), 1)
        dqkv, delta = self.new(T, 3 * a), self.f32(self.heads * T)
        n = L.mc_attention_backward_ws_bytes(B, S, self.heads, self.d)
        self.run(L.mc_attention_backward_ws(self.qkv, self.o, self.lse, do, dqkv, delta, B, S, self.heads,
                                            self.d, self.new(n, dtype=torch.uint8), n, self.st,
                                            torch.cuda.current_stream()))
        if self.norm is not None:
            names = [x + y for y in ("_gain", "_shift") for x in "qk"]
            sums = [None if x is None else self.f32(self.d) for x in
                    (self.norm.tensors[i] for i in (0, 2, 1, 3))]
            scratch = self.f32(L.mc_qk_norm_scratch_floats(T, self.heads, self.heads, self.d))
            self.run(L.mc_qk_norm_backward(self.raw, dqkv, dqkv, T, self.heads, self.heads, self.d, 2 * a,
                                           3 * a, 3 * a, self.norm,
                                           grads=L.make_qk_norm_grads(**dict(zip(names, sums))),
                                           scratch=scratch, status=self.st))
            for name, x in zip(("q_norm_g", "k_norm_g", "q_norm_b", "k_norm_b"), sums):
                if x is not None:
                    g[name] = x
        g["w_qkv"] = self.gemm(3 * a, HID, T, dqkv, 1, self.ln1, 1, self.f32(3 * a, HID), 0)
        dln = self.gemm(T, HID, 3 * a, dqkv, 0, w["w_qkv"], 1, self.f32(T, HID), 0)
        dx = self.norm_rows_back("ln1", dln, self.x, self.s1, dx1, None, None)
        return dx, g, {"b_fc2": dy, "b_fc1": dhp, "b_qkv": dqkv}


@pytest.mark.parametrize("kind", ["none", "plain", "gains", "centred"])
@pytest.mark.parametrize("heads,d", [(4, 64), (2, 128)])
def test_the_parts_bits(heads, d, kind):
    params, x, dy = inputs(heads, d)
    norm = make_norm(kind, d)
    layer = TransformerLayer(B, S, HID, heads, F, head_dim=d, params=params, qk_norm=norm)
    y, dx = layer.forward(x), layer.backward(dy)
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    parts = Parts(params, heads, d, norm)
    assert torch.equal(parts.forward(x), y)
    want, grads, columns = parts.backward(dy)
    check_status(parts.st)
    assert torch.equal(dx, want)
    assert set(layer.grads) == set(grads) | set(columns)
    for name, g in grads.items():
        assert torch.equal(layer.grads[name], g), name
    for name, rows in columns.items():
        # sums of 304 numbers in 32 bits: each partial sum is off by half a step of at
        # most the sum of the sizes, 304 2^-24 < 2^-15 of it
        rows = rows.double()
        off = (layer.grads[name].double() - rows.sum(0)).abs()
        assert (off <= 2.0 ** -15 * rows.abs().sum(0)).all(), name


@pytest.mark.parametrize("kind", ["plain", "gains", "centred"])
def test_heads_of_128_against_float64(monkeypatch, kind):
    heads, d = 2, 128
    monkeypatch.setattr(N, "H", heads)
    monkeypatch.setattr(N, "D", d)
    params, x, dy = inputs(heads, d)
    norm = make_norm(kind, d)
    layer = TransformerLayer(B, S, HID, heads, F, head_dim=d, params=params, qk_norm=norm)
    y, dx = layer.forward(x), layer.backward(dy)
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    w = {n: v.detach().double().cpu().requires_grad_() for n, v in params.items()}
    n64 = [None if t is None else t.double().cpu().requires_grad_() for t in norm.tensors]
    ones = torch.ones(d, dtype=torch.float64)
    used = [ones if t is None and i % 2 == 0 else t for i, t in enumerate(n64)]
    # (a zero for every key's shift: its gradient holds the terms of the shift's)
    each = torch.zeros(B, heads, S, d, dtype=torch.float64, requires_grad=True)
    if used[3] is not None:
        used[3] = used[3] + each
    x64 = x.double().cpu().view(B, S, HID).requires_grad_()
    lo, hi = torch.zeros(B, S, dtype=torch.int64), torch.arange(1, S + 1).expand(B, S)
    y64 = N.torch_layer(x64, w, norm, used, None, lo, hi)
    y64.backward(dy.double().cpu().view(B, S, HID))
    assert_close("y", to_f64(y), y64.detach().numpy().reshape(T, HID), *N.TOL)
    assert_close("dx", to_f64(dx), x64.grad.numpy().reshape(T, HID), *N.TOL)
    for n in w:
        assert_close(n, to_f64(layer.grads[n]), w[n].grad.numpy(), *N.TOL)
    # (the norms' gradients: ten roundings of either sign, as with heads of 64)
    for n, t in zip(N.NAMES, n64):
        assert (n in layer.grads) == (t is not None)
        if n == "k_norm_b" and t is not None:
            # A number added to all of a row's scores leaves the softmax as it is, so
            # without a rotation the keys' shift has the gradient 0: sums over tokens and
            # heads of terms that cancel.  What is left are the terms' roundings, ten of
            # either sign, at most 2^-8 of the term each: sqrt(10) 2^-8 of the 2-norm of
            # all terms in the 2-norm of the sums.
            assert t.grad.abs().max() <= 1e-12 * each.grad.abs().max()
            assert layer.grads[n].double().norm().item() <= math.sqrt(10) * 2.0 ** -8 * each.grad.norm()
        elif t is not None:
            m = metrics(to_f64(layer.grads[n]), t.grad.numpy())
            assert m["finite"] and m["max_rel"] <= N.TOL[0] and \
                m["norm_rel"] <= math.sqrt(10) * 2.0 ** -8, (n, m)
