"""Which gradients of its norms a layer offers after they were exchanged: those that
its present norm has, none with what an earlier one left."""
import pytest
import torch

from megatron_transformer_layer_gb300 import _lib as L
from megatron_transformer_layer_gb300.layer import TransformerLayer

P = 1 << 20  # a pointer that is aligned and never dereferenced
NAMES = ("q_norm_g", "q_norm_b", "k_norm_g", "k_norm_b")


def offered(layer):
    return [n for n in NAMES if n in layer.grads]


def test_entries_follow_the_norm(monkeypatch):
    monkeypatch.setattr(L, "make_qk_norm_grads", lambda *a: L.mc_qk_norm_grads())
    layer = TransformerLayer(1, 64, 128, 2, 256, device="cpu", qk_norm=L.make_qk_norm(P, P, P, P))
    assert offered(layer) == list(NAMES)
    others = [n for n in layer.grads if n not in NAMES]
    layer.set_qk_norm(L.make_qk_norm(P, P))
    assert offered(layer) == ["q_norm_g", "k_norm_g"]
    layer.set_qk_norm(L.make_qk_norm(None, P, P))
    assert offered(layer) == ["q_norm_b", "k_norm_g"]
    layer.set_qk_norm(L.make_qk_norm())
    assert offered(layer) == [] and list(layer.grads) == others
    layer.set_qk_norm(L.make_qk_norm(P, P, P, P))
    assert offered(layer) == list(NAMES)


def test_a_structure_of_bare_pointers():
    """Filled field by field, as a C program would: the library's own checks come first."""
    n = L.mc_layer_qk_norm(L.mc_qk_norm(P, None, P, None, 0.0, 0))
    sh = L.make_shape(1, 64, 768, 12, 2304)
    rc = L.mc_layer_forward_norm(sh, L.mc_layer_weights(*[P] * 12), n, None, None, P, P, P, P, 1 << 40)
    assert rc == L.MC_ERR_ARGUMENT  # (eps)


@pytest.mark.gpu
@pytest.mark.parametrize("accumulate", [False, True])
def test_no_gradient_of_an_earlier_norm(accumulate):
    """From shifts to none and back: the values are those of a layer that was built so."""
    from gpu_util import DEV
    from test_gpu_attention_opt import gen
    from test_gpu_layer_qk_norm import B, F, H, HID, T, make_norm
    params = TransformerLayer.random_params(HID, H, F, seed=3, std=0.05)
    x, dy = (torch.randn(T, HID, generator=gen(k)).to(DEV) for k in (1, 2))
    S = T // B

    def step(layer):
        layer.forward(x)
        layer.backward(dy)
        torch.cuda.synchronize()
        return {n: layer.grads[n].clone() for n in offered(layer)}

    def built(norm):
        return TransformerLayer(B, S, HID, H, F, params=params, qk_norm=norm,
                                accumulate_grads=accumulate)

    shifts, plain = make_norm(True), make_norm(True, shifts=False)
    want = {id(n): step(built(n)) for n in (shifts, plain)}
    layer = built(shifts)
    for norm in (shifts, plain, shifts):
        layer.set_qk_norm(norm)
        for g in layer.grads.values():
            g.zero_()
        got = step(layer)
        assert list(got) == list(want[id(norm)])
        assert all(torch.equal(got[n], want[id(norm)][n]) for n in got)


@pytest.mark.gpu
def test_a_gradient_that_comes_back_starts_at_zero():
    from gpu_util import DEV
    from test_gpu_attention_opt import gen
    from test_gpu_layer_qk_norm import B, F, H, HID, T, make_norm
    params = TransformerLayer.random_params(HID, H, F, seed=3, std=0.05)
    layer = TransformerLayer(B, T // B, HID, H, F, params=params, qk_norm=make_norm(True),
                             accumulate_grads=True)
    x, dy = (torch.randn(T, HID, generator=gen(k)).to(DEV) for k in (1, 2))
    layer.forward(x)
    layer.backward(dy)
    kept = layer.grads["q_norm_g"].clone()
    layer.set_qk_norm(make_norm(True, shifts=False))
    layer.set_qk_norm(make_norm(True))
    torch.cuda.synchronize()
    assert torch.equal(layer.grads["q_norm_g"], kept) and bool(kept.any())  # (never left)
    assert not layer.grads["q_norm_b"].any() and not layer.grads["k_norm_b"].any()
