"""The index and constant arrays of positions and masks, given as tensors: what
the binding refuses before a pointer reaches the library.  (Without a GPU the
last thing it finds is that the tensors are not on one.)"""
import pytest
import torch

from megatron_transformer_layer_gb300 import _lib as L

P = 1 << 20  # a pointer that is aligned and never dereferenced
B, S = 2, 300
ROWS, INTS = B * S, L.mc_attention_mask_table_ints(B, S)
X = torch.zeros(4, 128, dtype=torch.bfloat16)
SPEC = L.make_rotary_spec(64, [16, 8, 8])


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def documents(offsets=P, n=3, prefix=P, key_lo=P, key_hi=P, tables=P):
    return L.mc_attention_mask_documents(offsets, n, prefix, 1, 0, B, S, key_lo, key_hi, tables)


def given(key_lo=P, key_hi=P, tables=P):
    return L.mc_attention_mask_intervals(B, S, key_lo, key_hi, tables)


def rotary(positions=P, inv_freq=P):
    return L.mc_rotary_forward(X, X, 4, 2, 64, 128, 128, positions, inv_freq, SPEC)


def rotary_back(positions=P, inv_freq=P):
    return L.mc_rotary_backward(X, X, 4, 2, 64, 128, 128, positions, inv_freq, SPEC)


def layer_rotary(positions=P, inv_freq=P):
    return L.make_layer_rotary(SPEC, positions, inv_freq)


def options(key_lo=P, key_hi=P, tables=P, slopes=P):
    return L.make_attention_options(key_lo, key_hi, tables, slopes)


ARRAYS = [(documents, "offsets", torch.int32, 4), (documents, "prefix", torch.int32, 3),
          (documents, "key_lo", torch.int32, ROWS), (documents, "key_hi", torch.int32, ROWS),
          (documents, "tables", torch.int32, INTS), (given, "key_lo", torch.int32, ROWS),
          (given, "key_hi", torch.int32, ROWS), (given, "tables", torch.int32, INTS),
          (rotary, "positions", torch.int32, 12), (rotary, "inv_freq", torch.float32, 32),
          (rotary_back, "positions", torch.int32, 12), (rotary_back, "inv_freq", torch.float32, 32),
          (layer_rotary, "positions", torch.int32, 0), (layer_rotary, "inv_freq", torch.float32, 32),
          (options, "key_lo", torch.int32, 0), (options, "key_hi", torch.int32, 0),
          (options, "tables", torch.int32, 0), (options, "slopes", torch.float32, 0)]


@pytest.mark.parametrize("call,name,dtype,n", ARRAYS)
def test_arrays_are_checked(call, name, dtype, n):
    for other in (torch.int64, torch.int16, torch.float64, torch.bfloat16, torch.float32,
                  torch.int32):
        if other is not dtype:
            with pytest.raises(TypeError, match=name):
                call(**{name: torch.zeros(n + 8, dtype=other)})
    with pytest.raises(ValueError, match=f"{name}.*contiguous"):
        call(**{name: torch.zeros(2 * n + 8, dtype=dtype)[::2]})
    with pytest.raises(ValueError, match=f"{name}.*contiguous"):
        call(**{name: torch.zeros(1, dtype=dtype).expand(n + 8)})
    if n:
        with pytest.raises(ValueError, match=f"{name}.*{n} elements"):
            call(**{name: torch.zeros(n - 1, dtype=dtype)})
    with pytest.raises(ValueError, match=f"{name}.*on the GPU"):
        call(**{name: torch.zeros(n + 8, dtype=dtype)})


def test_one_text_position_expanded_over_axes():
    with pytest.raises(ValueError, match="positions.*contiguous"):
        rotary(positions=i32(1, 4).expand(3, -1))


@pytest.mark.parametrize("lengths,name", [((ROWS - 1, INTS, 2), "key_lo"),
                                          ((ROWS, INTS - 8, 2), "tables"),
                                          ((ROWS, INTS, 1), "slopes")])
def test_options_of_another_shape(lengths, name):
    """Lengths are compared with each call's shape: the layer's too."""
    opt = options()
    opt.lengths = lengths
    sh = L.make_shape(B, S, 128, 2, 256)
    w, g = L.mc_layer_weights(*[P] * 12), L.mc_layer_grads(*[P] * 12)
    for call in (lambda: L.mc_attention_forward_opt(P, P, P, B, S, 2, 64, opt),
                 lambda: L.mc_attention_backward_opt(P, P, P, P, P, P, B, S, 2, 64, opt),
                 lambda: L.mc_layer_forward_opt(sh, w, None, opt, P, P, P, P, 0),
                 lambda: L.mc_layer_backward_opt(sh, w, None, opt, P, P, P, P, g, P, 0)):
        with pytest.raises(ValueError, match=name):
            call()
    opt.lengths = (ROWS, INTS, 2)   # enough: the library's own checks come next
    assert L.mc_attention_forward_opt(None, P, P, B, S, 2, 64, opt) == L.MC_ERR_NULLPTR
    assert L.mc_layer_forward_opt(sh, w, None, opt, P, P, P, P, 0) == L.MC_ERR_WORKSPACE


def test_positions_of_fewer_tokens_than_the_layer():
    sh = L.make_shape(B, S, 128, 2, 256)
    w, g = L.mc_layer_weights(*[P] * 12), L.mc_layer_grads(*[P] * 12)
    rot = layer_rotary()
    rot.length = 3 * ROWS - 1
    for call in (lambda: L.mc_layer_forward_opt(sh, w, rot, None, P, P, P, P, 0),
                 lambda: L.mc_layer_backward_opt(sh, w, rot, None, P, P, P, P, g, P, 0)):
        with pytest.raises(ValueError, match="positions"):
            call()
    rot.length = 3 * ROWS
    assert L.mc_layer_forward_opt(sh, w, rot, None, P, P, P, P, 0) == L.MC_ERR_WORKSPACE


def test_none_and_pointers_go_to_the_librarys_checks():
    assert documents(offsets=None) == L.MC_ERR_NULLPTR
    assert given(tables=P + 4) == L.MC_ERR_ALIGN
    assert rotary(positions=None) == L.MC_ERR_NULLPTR
