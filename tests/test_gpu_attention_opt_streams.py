"""The binding's calls of positions and masks without a stream argument go to
torch's current stream, as the layer's do: what a program makes on a side stream
is read there.  Shown by capturing them: a call on another stream would not be
in the graph."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_gb300 import _lib as L
from megatron_transformer_layer_gb300.layer import TransformerLayer

from gpu_util import DEV, check_status, status
from test_gpu_attention_opt import bf16, gen, i32

pytestmark = pytest.mark.gpu

B, S, H, D = 1, 300, 2, 64
A = H * D


def replayed(call, outputs):
    """outputs after `call` on the current stream, and after its replay."""
    codes = call()
    assert codes == [0] * len(codes)
    torch.cuda.synchronize()
    want = [x.clone() for x in outputs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    torch.cuda.synchronize()
    for x in outputs:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    return want, outputs


def same(pair):
    return all(torch.equal(x, y) for x, y in zip(*pair))


def test_calls_without_a_stream():
    st = status()
    lo, hi, lo2, hi2 = (torch.empty(B, S, dtype=torch.int32, device=DEV) for _ in range(4))
    n = L.mc_attention_mask_table_ints(B, S)
    tab, tab2 = torch.empty(n, dtype=torch.int32, device=DEV), torch.empty(n, dtype=torch.int32,
                                                                           device=DEV)
    off, pos = i32([0, 100, 300]), i32(np.arange(S)[None])
    assert same(replayed(lambda: [L.mc_attention_mask_documents(off, 2, None, 1, 0, B, S, lo, hi,
                                                                tab, st)], [lo, hi, tab]))
    lo2.copy_(lo), hi2.copy_(hi)
    assert same(replayed(lambda: [L.mc_attention_mask_intervals(B, S, lo2, hi2, tab2, st)], [tab2]))
    qkv, dout = bf16(gen(1), B * S, 3 * A), bf16(gen(2), B * S, A)
    turned, back, dqkv = (torch.zeros_like(qkv) for _ in range(3))
    freq, spec = torch.rand(32, generator=gen(3)).to(DEV), L.make_rotary_spec(64)
    a = (S, 2 * H, D, 3 * A, 3 * A, pos, freq, spec, st)
    assert same(replayed(lambda: [L.mc_rotary_forward(qkv, turned, *a),
                                  L.mc_rotary_backward(turned, back, *a)], [turned, back]))
    opt = L.make_attention_options(lo, hi, tab)
    o, lse = torch.empty(S, A, dtype=torch.bfloat16, device=DEV), torch.empty(H * S, device=DEV)
    delta, ws = torch.empty(H * S, device=DEV), torch.empty(
        L.mc_attention_backward_opt_ws_bytes(B, S, H, D, opt), dtype=torch.uint8, device=DEV)
    shape = (B, S, H, D, opt)
    assert same(replayed(lambda: [L.mc_attention_forward_opt(qkv, o, lse, *shape, st)], [o, lse]))
    assert same(replayed(lambda: [L.mc_attention_backward_opt(qkv, o, lse, dout, dqkv, delta, *shape,
                                                              ws, ws.numel(), st)], [dqkv]))
    check_status(st)


def test_layer_calls_without_a_stream():
    params = TransformerLayer.random_params(128, H, 256, seed=5)
    layer = TransformerLayer(B, S, 128, H, 256, params=params)
    x, dy = torch.randn(S, 128, generator=gen(1)).to(DEV), torch.randn(S, 128,
                                                                       generator=gen(2)).to(DEV)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    lo, hi = i32(np.zeros((B, S))), i32(np.arange(1, S + 1)[None])
    tab = torch.empty(L.mc_attention_mask_table_ints(B, S), dtype=torch.int32, device=DEV)
    assert L.mc_attention_mask_intervals(B, S, lo, hi, tab) == 0
    opt = L.make_attention_options(lo, hi, tab)
    w = (layer.shape, layer.weights, None, opt)
    assert same(replayed(
        lambda: [L.mc_layer_forward_opt(*w, x, y, layer.saved, layer.ws, layer.ws_bytes),
                 L.mc_layer_backward_opt(*w, x, dy, layer.saved, dx, layer._grads_c, layer.ws,
                                         layer.ws_bytes)], [y, dx]))
    assert layer.device_status() == 0


def test_an_explicit_stream_still_counts():
    lo, hi = i32(np.zeros((B, S))), i32(np.arange(1, S + 1)[None])
    tab = torch.zeros(L.mc_attention_mask_table_ints(B, S), dtype=torch.int32, device=DEV)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        assert L.mc_attention_mask_intervals(B, S, lo, hi, tab, None, side) == 0
    side.synchronize()
    assert tab.any()
