"""The layer with norms of its queries and keys under shape flags together."""
import pytest
import torch

from megatron_transformer_layer_gb300.layer import TransformerLayer

from gpu_util import DEV, to_f64
from parity import assert_close
from test_gpu_attention_opt import gen
from test_gpu_layer_qk_norm import B, F, H, HID, S, T, TOL, make_norm

pytestmark = pytest.mark.gpu


def step(**flags):
    params = TransformerLayer.random_params(HID, H, F, seed=3, std=0.05)
    layer = TransformerLayer(B, S, HID, H, F, 2, params=params, qk_norm=make_norm(True), **flags)
    x, dy = (torch.randn(T, HID, generator=gen(k)).to(DEV) for k in (1, 2))
    for _ in range(2):
        y, dx = layer.forward(x), layer.backward(dy)
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    return dict(layer.grads, y=y, dx=dx)


@pytest.mark.parametrize("flags", [dict(), dict(fp8=True), dict(attn_dq_recompute=True),
                                   dict(sequence_parallel=True, accumulate_grads=True),
                                   dict(fp8=True, accumulate_grads=True, attn_dq_recompute=True)])
def test_recomputed_activations_keep_the_bits(flags):
    a, b = step(**flags), step(recompute=True, **flags)
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("flags,times", [(dict(attn_dq_recompute=True), 1),
                                         (dict(sequence_parallel=True, accumulate_grads=True), 2)])
def test_the_same_gradients(flags, times):
    a, b = step(), step(**flags)
    assert set(a) == set(b)
    for n in a:
        assert_close(n, to_f64(b[n]), to_f64(a[n]) * (1 if n in ("y", "dx") else times), *TOL)
