"""What the binding refuses of the tensors that the norms of queries and keys read and
write, before anything is launched: those on another device, of another type, with
fewer rows or elements than the call covers, or of another stride than it states."""
import pytest
import torch

from megatron_transformer_layer_gb300 import _lib as L

T, QH, KH, D = 4, 2, 1, 64
W = (QH + KH) * D
NORM = L.make_qk_norm()


class Fake(torch.Tensor):
    """A CPU tensor that says it is on the GPU: nothing here may reach a launch."""

    is_cuda = True


def fake(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Fake)


@pytest.fixture
def launched(monkeypatch):
    """Calls that passed the binding's checks, instead of the library."""
    seen = []

    class Library:
        @staticmethod
        def mc_qk_norm_forward(*a):
            seen.append(a)
            return 0

        mc_qk_norm_backward = mc_qk_norm_forward
        mc_qk_norm_scratch_floats = staticmethod(lambda *a: 0)
    monkeypatch.setattr(L, "lib", lambda: Library)
    monkeypatch.setattr(L, "_on", lambda stream, x: None)
    return seen


def forward(x, out, ld_in=W, ld_out=W, tokens=T):
    return L.mc_qk_norm_forward(x, out, tokens, QH, KH, D, ld_in, ld_out, NORM)


def backward(x, dout, din, lds=(W, W, W), tokens=T):
    return L.mc_qk_norm_backward(x, dout, din, tokens, QH, KH, D, *lds, NORM)


def wide(extra=8, **kw):
    return fake(T, W + extra, **kw)


@pytest.mark.parametrize("good", [
    (lambda: fake(T, W), W), (lambda: wide(), W + 8), (lambda: wide()[:, 4:], W + 8),
    (lambda: fake(T + 3, W), W), (lambda: fake(T, QH + KH, D), W), (lambda: fake(T * (QH + KH), D), W),
    (lambda: fake(2, T // 2, QH + KH, D), W), (lambda: fake(T * W), W),
    (lambda: fake(T, 3, QH + KH, D)[:, 1], 3 * W),
    (lambda: fake(T * (W + 1) + 1)[1:].view(T, W + 1), W + 1),
    (lambda: fake(T, W, dtype=torch.float32), W)])
def test_rows_that_cover_the_call(launched, good):
    make, ld = good
    x = make()
    assert forward(x, x, ld, ld) == 0 and backward(x, x, x, (ld,) * 3) == 0
    assert len(launched) == 2 and launched[0][0] == x.data_ptr()


def test_one_row_has_no_stride(launched):
    x = fake(9, W)[::2][:1]
    assert forward(x, x, W, W, 1) == 0 and len(launched) == 1


@pytest.mark.parametrize("bad,message", [
    (lambda: torch.zeros(T, W, dtype=torch.bfloat16), "on the GPU"),
    (lambda: fake(T - 1, W), "4 rows of 192"),
    (lambda: fake(T, W - 1), "4 rows of 192"),
    (lambda: wide(), "192 apart"),              # another stride than stated
    (lambda: wide()[:, :W], "192 apart"),
    (lambda: fake(W, T).t(), "4 rows of 192"),  # columns
    (lambda: fake(T, 2 * W)[:, ::2], "4 rows of 192"),
    (lambda: fake(T * W - 1), "4 rows of 192"),
    (lambda: fake(T, QH, D), "4 rows of 192"),
    (lambda: fake(T, 3, QH + KH, D)[:, 1], "192 apart"),
    (lambda: fake(T, 3, QH, D)[:, 1], "192 apart")])
def test_rows_that_do_not(launched, bad, message):
    x, good = bad(), fake(T, W)
    calls = [lambda: forward(x, good), lambda: forward(good, x), lambda: backward(x, good, good),
             lambda: backward(good, x, good), lambda: backward(good, good, x)]
    for call, name in zip(calls, ("x", "out", "x", "dout", "din")):
        with pytest.raises(ValueError, match=f"^{name}: .*{message}"):
            call()
    assert not launched


def test_types(launched):
    x = fake(T, W, dtype=torch.float16)
    for call in (lambda: forward(x, x), lambda: backward(x, x, x)):
        with pytest.raises(TypeError, match="norms of queries and keys take bf16 or fp32"):
            call()
    assert not launched


def test_rotary_positions_say_their_own_name():
    x = torch.zeros(4, 64, dtype=torch.float16)
    with pytest.raises(TypeError, match="rotary positions take bf16 or fp32"):
        L.mc_rotary_forward(x, x, 4, 1, 64, 64, 64, None, None, L.make_rotary_spec(64))
