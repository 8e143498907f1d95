"""The largest calls of the attention to keys of another length that are taken, without
a GPU: how many blocks of queries or keys a call may count."""
import pytest

from megatron_transformer_layer_gb300 import _lib as L

from test_cross_attention_host import P, cross_calls


def call(n, rows, heads, **kw):
    return L.make_cross_attention(n, rows, rows, heads, heads, 64, q_offsets=P, kv_offsets=P, **kw)


@pytest.mark.parametrize("n,rows,heads", [(1 << 18, 512, 1024), (1 << 20, 128, 1024), (1 << 20, 1, 1024)])
def test_items_are_below_2_to_the_30(n, rows, heads):
    """Twice as many have to be a 32-bit number."""
    c = call(n, rows, heads)
    assert cross_calls(c) == (L.MC_ERR_UNSUPPORTED,) * 2
    assert L.mc_attention_backward_cross_ws_bytes(c) == 0
    assert L.mc_attention_backward_cross_ws_bytes(call(n - 1, rows, heads)) > 0
