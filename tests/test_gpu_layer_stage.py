"""The layer's attention stage: positions without a mask, a mask without
positions, and both changed from batch to batch (set_stage).  And angles of
frequencies far from one, which the fixed-point turns have to hold."""
import numpy as np
import pytest
import torch

import oracle.attention_opt as O
from megatron_transformer_layer_gb300 import _lib as L
from megatron_transformer_layer_gb300.layer import TransformerLayer

from gpu_util import DEV, check_status, status, to_f64
from parity import assert_close
from test_gpu_attention_opt import gen, make_documents, torch_layer

pytestmark = pytest.mark.gpu

B, S, HID, H, F, D = 2, 152, 256, 4, 512, 64
T = B * S
TOL = (2e-2, 2e-3)  # the layer's own gate


def make_rotary():
    pos = torch.randint(0, 400, (1, T), generator=gen(11), dtype=torch.int32)
    freq = torch.rand(32, generator=gen(12))
    return (64, [0] * 32, pos, freq), \
        L.make_layer_rotary(L.make_rotary_spec(64), pos.to(DEV), freq.to(DEV))


def causal():
    lo, hi = np.zeros((B, S), dtype=np.int64), np.tile(np.arange(1, S + 1), (B, 1))
    return torch.from_numpy(lo), torch.from_numpy(hi)


def make_mask(ahead=False, off=(0, 40, 152, 250, 300)):
    pre = [10, 30, 0, 20] if ahead else None
    lo, hi, tab = make_documents(list(off), pre, True, 0, B, S)
    return (lo.cpu().long(), hi.cpu().long()), L.make_attention_options(lo, hi, tab, None, 8.0,
                                                                        causal=not ahead)


def inputs():
    return torch.randn(T, HID, generator=gen(1)).to(DEV), torch.randn(T, HID, generator=gen(2)).to(DEV)


def step(layer, x, dy):
    y, dx = layer.forward(x), layer.backward(dy)
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    return [t.clone() for t in (y, dx, *layer.grads.values())]


@pytest.mark.parametrize("with_rotary,with_mask", [(True, False), (False, True)])
@pytest.mark.parametrize("flags", [dict(), dict(recompute=True)])
def test_layer_with_one_of_them(with_rotary, with_mask, flags):
    params = TransformerLayer.random_params(HID, H, F, seed=3, std=0.05)
    ref_rot, rot = make_rotary() if with_rotary else (None, None)
    (lo, hi), att = make_mask() if with_mask else (causal(), None)
    layer = TransformerLayer(B, S, HID, H, F, 2, params=params, rotary=rot, attention=att, **flags)
    x, dy = inputs()
    y, dx, *_ = step(layer, x, dy)
    w = {n: v.detach().double().cpu().requires_grad_() for n, v in params.items()}
    x64 = x.double().cpu().view(B, S, HID).requires_grad_()
    y64 = torch_layer(x64, w, H, D, None, ref_rot, lo, hi, None, 8.0 if with_mask else 0.0)
    y64.backward(dy.double().cpu().view(B, S, HID))
    assert_close("y", to_f64(y), y64.detach().numpy().reshape(T, HID), *TOL)
    assert_close("dx", to_f64(dx), x64.grad.numpy().reshape(T, HID), *TOL)
    for n in w:
        assert_close(n, to_f64(layer.grads[n]), w[n].grad.numpy(), *TOL)


def test_set_stage():
    """A layer whose stage is set gives the bits of one built with it, whatever
    ran before; what its workspace does not cover is refused and changes
    nothing."""
    params = TransformerLayer.random_params(HID, H, F, seed=3, std=0.05)
    x, dy = inputs()

    def built(**stage):
        return TransformerLayer(B, S, HID, H, F, params=params, **stage)

    _, rot = make_rotary()
    masks = [make_mask()[1], make_mask(off=(0, 100, 101, 152, 304))[1]]
    _, ahead = make_mask(ahead=True)
    want = [step(built(), x, dy), step(built(rotary=rot), x, dy)] + \
        [step(built(rotary=rot, attention=m), x, dy) for m in masks]
    layer = built()
    for stage, w in zip(((), (rot,), (rot, masks[0]), (rot, masks[1]), ()), want + want[:1]):
        layer.set_stage(*stage)
        assert all(torch.equal(u, v) for u, v in zip(step(layer, x, dy), w))
    with pytest.raises(L.McError):
        layer.set_stage(rot, ahead)
    assert all(torch.equal(u, v) for u, v in zip(step(layer, x, dy), want[0]))
    # built for a mask that looks ahead: covers the others too
    layer = built(attention=ahead)
    seen = step(layer, x, dy)
    layer.set_stage(rot, masks[1])
    assert all(torch.equal(u, v) for u, v in zip(step(layer, x, dy), want[3]))
    layer.set_stage(attention=ahead)
    assert all(torch.equal(u, v) for u, v in zip(step(layer, x, dy), seen))


def test_set_stage_of_too_few_positions():
    layer = TransformerLayer(B, S, HID, H, F, params=TransformerLayer.random_params(HID, H, F))
    short = torch.zeros(1, T - 1, dtype=torch.int32, device=DEV)
    layer.set_stage(L.make_layer_rotary(L.make_rotary_spec(64), short, torch.ones(32, device=DEV)))
    with pytest.raises(ValueError, match="positions"):
        layer.forward(inputs()[0])


@pytest.mark.parametrize("inverse", [False, True])
def test_rotary_frequencies_far_from_one(inverse):
    freq = torch.tensor([0.0, -0.0, 1e-45, 2.0 ** -126, 1e-30, 2.0 ** -64, 2.0 ** -33, -3e-9, -0.7,
                         1.0, 3.1415927, 6.2831855, -100.0, 1e4, 2.0 ** 24 + 2, 3e7, 1e12, -1e15,
                         2.0 ** 31, 2.0 ** 40])
    n, tokens = freq.numel(), 40
    g = gen(7)
    x = torch.randn(tokens, 2 * n, generator=g).to(DEV)
    pos = torch.randint(-(2 ** 31), 2 ** 31, (1, tokens), generator=g).to(torch.int32)
    pos[0, :6] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -(2 ** 31), 12345])
    ref = O.rotary(to_f64(x).reshape(tokens, 1, 2 * n), pos.numpy(), freq.numpy(), 2 * n, [n],
                   inverse=inverse).reshape(tokens, -1)
    # the result's rounding, and as in test_rotary 2^-20 for the angle (2^-33 of
    # a turn from the fixed point, 2^-25 of half a turn from its 32-bit float)
    tol = 2.0 ** -24 * np.abs(ref) + np.abs(to_f64(x)).max() * 2.0 ** -20
    out, st = torch.empty_like(x), status()
    call = L.mc_rotary_backward if inverse else L.mc_rotary_forward
    assert call(x, out, tokens, 1, 2 * n, 2 * n, 2 * n, pos.to(DEV), freq.to(DEV),
                L.make_rotary_spec(2 * n), st) == 0
    check_status(st)
    assert (np.abs(to_f64(out) - ref) <= tol).all()
