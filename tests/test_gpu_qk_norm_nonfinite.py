"""A NaN or an infinity in one head, of the input or of the gradient, stays there: every
other head, and the gradients of the other type's gain and shift, keep their bits."""
import pytest
import torch

from megatron_transformer_layer_gb300 import _lib as L

from gpu_util import DEV
from test_gpu_qk_norm import KEEP, Problem, check_status, status

pytestmark = pytest.mark.gpu

CASES = [dict(tokens=5, q_heads=3, k_heads=2, d=64, rot=64, centred=True),
         dict(tokens=7, q_heads=2, k_heads=1, d=128),
         dict(tokens=9, q_heads=3, k_heads=2, d=72, rot=48, adjacent=True),
         dict(tokens=6, q_heads=2, k_heads=2, d=96, rot=60, adjacent=True, extra=2),
         dict(tokens=6, q_heads=2, k_heads=2, d=7, rot=4, centred=True, dtype=torch.float32)]


def run(p):
    T, w = p.tokens, p.H * p.d
    out, st = torch.empty(T, w, dtype=p.dtype, device=DEV), status()
    assert L.mc_qk_norm_forward(p.x, out, *p.heads(), p.ld, w, p.norm, p.positions, p.inv_freq, p.spec,
                                st) == 0
    check_status(st)
    g = torch.full((4, p.d), KEEP, device=DEV)
    din = p.backward(L.make_qk_norm_grads(q_gain=g[0], q_shift=g[1], k_gain=g[2], k_shift=g[3]))
    return out.view(T, p.H, p.d), din.reshape(T, p.H, p.d), g


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("into", ["x", "dout"])
@pytest.mark.parametrize("case", CASES)
def test_stays_in_its_head(case, into, value):
    p = Problem(**case)
    want = run(p)
    # in the first token's first head of the keys, and in the last one's last
    where = [(0, p.q_heads), (p.tokens - 1, p.H - 1)]
    for t, h in where:
        getattr(p, into)[t, h * p.d + p.d // 2] = value
    got = run(p)
    others = torch.ones(p.tokens, p.H, dtype=torch.bool, device=DEV)
    for t, h in where:
        others[t, h] = False
    for a, b in zip(got[:2], want):
        assert torch.equal(a[others], b[others])
    assert torch.equal(got[2][:2], want[2][:2])
    assert not torch.isfinite(got[2][2]).all()
