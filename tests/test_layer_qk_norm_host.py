"""The layer with norms of its queries and keys, without a GPU: sizes, and what its
entry points and the binding refuse before anything is launched."""
import pytest

from megatron_transformer_layer_gb300 import _lib as L

P = 1 << 20  # a pointer that is aligned and never dereferenced


def shape(**kw):
    return L.make_shape(1, 64, 768, 12, 2304, **kw)


def norm(q_gain=None, grads=None, **kw):
    return L.make_layer_qk_norm(L.make_qk_norm(q_gain, **kw), grads)


def calls(sh, n, **change):
    a = dict(x=P, y=P, dy=P, dx=P, saved=P, ws=P, rotary=None, attention=None,
             ws_bytes=L.mc_layer_workspace_bytes_norm(sh, n, change.get("attention")))
    a.update(change)
    w, g = L.mc_layer_weights(*[P] * 12), L.mc_layer_grads(*[P] * 12)
    stage = (sh, w, n, a["rotary"], a["attention"], a["x"])
    return (L.mc_layer_forward_norm(*stage, a["y"], a["saved"], a["ws"], a["ws_bytes"]),
            L.mc_layer_backward_norm(*stage, a["dy"], a["saved"], a["dx"], g, a["ws"], a["ws_bytes"]))


def test_sizes():
    sh, n = shape(), norm()
    # Q | K as they were before their norms
    assert L.mc_layer_saved_bytes_norm(sh, n) == L.mc_layer_saved_bytes(sh) + 64 * 2 * 768 * 2
    assert L.mc_layer_saved_bytes_norm(sh, None) == L.mc_layer_saved_bytes(sh)
    assert L.mc_layer_workspace_bytes_norm(sh, None, None) == L.mc_layer_workspace_bytes(sh)
    assert L.mc_layer_workspace_bytes_norm(sh, n, None) >= L.mc_layer_workspace_bytes(sh)
    again = shape(flags=L.MC_RECOMPUTE_ACTIVATIONS)
    assert L.mc_layer_workspace_bytes_norm(again, n, None) >= \
        L.mc_layer_workspace_bytes(again) + 64 * 2 * 768 * 2
    ahead = L.make_attention_options(P, P, P, causal=False)
    assert L.mc_layer_workspace_bytes_norm(sh, None, ahead) == \
        L.mc_layer_workspace_bytes_opt(sh, ahead)
    bad = L.make_shape(1, 64, 768, 7, 2304)
    assert L.mc_layer_saved_bytes_norm(bad, n) == L.mc_layer_workspace_bytes_norm(bad, n, None) == 0


@pytest.mark.parametrize("n,change,code", [
    (norm(eps=0.0), {}, L.MC_ERR_ARGUMENT), (norm(eps=float("inf")), {}, L.MC_ERR_ARGUMENT),
    (norm(P + 1), {}, L.MC_ERR_ALIGN),
    (norm(grads=L.make_qk_norm_grads(P + 2)), {}, L.MC_ERR_ALIGN),
    (norm(), dict(rotary=L.make_layer_rotary(L.make_rotary_spec(66), P, P)), L.MC_ERR_SHAPE),
    (norm(), dict(rotary=L.make_layer_rotary(L.make_rotary_spec(64), None, P)), L.MC_ERR_NULLPTR),
    (norm(), dict(attention=L.make_attention_options(P, P, P, softcap=-1.0)), L.MC_ERR_ARGUMENT),
    (norm(), dict(x=None), L.MC_ERR_NULLPTR), (norm(), dict(saved=None), L.MC_ERR_NULLPTR),
    (norm(), dict(ws=P + 16), L.MC_ERR_ALIGN),
])
def test_refusals(n, change, code):
    assert calls(shape(), n, **change) == (code, code)


@pytest.mark.parametrize("flags", [0, L.MC_RECOMPUTE_ACTIVATIONS])
def test_workspace_too_small(flags):
    sh, n = shape(flags=flags), norm()
    need = L.mc_layer_workspace_bytes_norm(sh, n, None)
    assert calls(sh, n, ws_bytes=need - 1) == (L.MC_ERR_WORKSPACE,) * 2


def test_flags():
    n = norm()
    n.norm.flags = 6
    assert calls(shape(), n) == (L.MC_ERR_ARGUMENT,) * 2
