"""Norms of queries and keys with their rotation on the GPU, against the float64
oracle.  Tolerances: half a step of the stored type, and 2^-18 of the size of a
result's terms for 32-bit arithmetic (at most 256 squares summed, a reciprocal
square root of 2^-22, an angle of 2^-23 and some ten products and sums), set
before the first run."""
import numpy as np
import pytest
import torch

import oracle.cross_attention as O
from megatron_transformer_layer_gb300 import _lib as L

from gpu_util import DEV, check_status, status, to_f64

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -18
KEEP = 7.0


class Problem:
    def __init__(self, tokens, q_heads, k_heads, d, rot=0, sections=None, adjacent=False, dealt=False,
                 dtype=torch.bfloat16, centred=False, gains=True, shifts=None, extra=0, eps=1e-5,
                 seed=0):
        g = torch.Generator().manual_seed(seed + tokens + d)
        H = q_heads + k_heads
        self.tokens, self.q_heads, self.k_heads, self.d, self.H = tokens, q_heads, k_heads, d, H
        self.centred, self.eps, self.dtype, self.ld = centred, eps, dtype, H * d + extra
        x = torch.randn(tokens, H, d, generator=g) * (0.1 + 3 * torch.rand(H, 1, generator=g)) + \
            torch.randn(H, 1, generator=g)
        rows = torch.full((tokens, self.ld), KEEP)
        rows[:, : H * d] = x.reshape(tokens, -1)
        self.x = rows.to(dtype).to(DEV)
        self.dout = torch.randn(tokens, H * d + 2 * extra, generator=g).to(dtype).to(DEV)
        vec = lambda at: (at + 0.3 * torch.randn(d, generator=g)).bfloat16().to(DEV)  # noqa: E731
        self.gains = (vec(1.0), vec(1.0)) if gains else (None, None)
        shifts = centred if shifts is None else shifts
        self.shifts = (vec(0.0), vec(0.0)) if shifts else (None, None)
        self.norm = L.make_qk_norm(*self.gains, *self.shifts, eps=eps, centred=centred)
        self.positions = self.inv_freq = self.spec = self.turn = None
        if rot:
            axes = len(sections) if sections else 1
            pos = torch.randint(-3, 5000, (axes, tokens), generator=g, dtype=torch.int32)
            pos[0, 0], pos[-1, -1] = 2 ** 31 - 1, -(2 ** 31)
            freq = torch.tensor([500000.0 ** (-2.0 * p / rot) for p in range(rot // 2)]).float()
            self.spec = L.make_rotary_spec(rot, sections, adjacent, dealt)
            self.turn = (pos.numpy(), freq.numpy(), rot, sections or [rot // 2], adjacent, dealt)
            self.positions, self.inv_freq = pos.to(DEV), freq.to(DEV)

    def heads(self):
        return self.tokens, self.q_heads, self.k_heads, self.d

    def f64(self, x):
        return None if x is None else to_f64(x)

    def oracle_args(self):
        return (to_f64(self.x)[:, : self.H * self.d].reshape(self.tokens, self.H, self.d),
                self.q_heads, self.k_heads, self.eps, self.centred,
                tuple(map(self.f64, self.gains)))

    def check_forward(self):
        T, w, d = self.tokens, self.H * self.d, self.d
        x, qh, kh, eps, centred, gains = self.oracle_args()
        shifts = tuple(map(self.f64, self.shifts))
        ref = O.qk_norm(x, qh, kh, eps, centred, gains, shifts, self.turn).reshape(T, w)
        flat = np.abs(O.qk_norm(x, qh, kh, eps, centred, gains, shifts))
        # where the mean is taken off, what it was taken off counts
        n, r = O._moments(x, eps, centred)
        lost = np.abs(x).max(axis=2, keepdims=True) * r * max(
            1.0, *[np.abs(v).max() for v in gains if v is not None], 1.0) if centred else 0.0
        size = np.broadcast_to(flat.max(axis=2, keepdims=True) + lost, flat.shape).reshape(T, w)
        tol = torch.finfo(self.dtype).eps / 2 * np.abs(ref) + F32 * size
        out = torch.full((T + 1, w + 5), KEEP, dtype=self.dtype, device=DEV)
        st = status()
        args = (self.norm, self.positions, self.inv_freq, self.spec, st)
        assert L.mc_qk_norm_forward(self.x, out, *self.heads(), self.ld, w + 5, *args) == 0
        check_status(st)
        got = to_f64(out)
        off = np.abs(got[:T, :w] - ref) / tol
        assert off.max() <= 1, f"{off.max():.3g} of the tolerance"
        assert (got[T:] == KEEP).all() and (got[:, w:] == KEEP).all()
        # in place, at an address and stride that only whole elements divide
        y = torch.full((T * (self.ld + 1) + 1,), KEEP, dtype=self.dtype, device=DEV)
        rows = y[1:].view(T, self.ld + 1)
        rows[:, : self.ld] = self.x
        assert L.mc_qk_norm_forward(rows, rows, *self.heads(), self.ld + 1, self.ld + 1, *args) == 0
        check_status(st)
        got = to_f64(rows)
        assert (np.abs(got[:, :w] - ref) <= tol).all()
        assert torch.equal(rows[:, w: self.ld], self.x[:, w:]) and (got[:, self.ld] == KEEP).all()
        assert float(y[0]) == KEEP
        return self

    def backward(self, grads, accumulate=0, in_place=False):
        T, w, d = self.tokens, self.H * self.d, self.d
        n = L.mc_qk_norm_scratch_floats(*self.heads())
        scratch = torch.full((n + 1,), KEEP, device=DEV)
        dout = self.dout.clone()
        din = dout if in_place else torch.full((T + 1, w + 8), KEEP, dtype=self.dtype, device=DEV)
        st = status()
        assert L.mc_qk_norm_backward(self.x, dout, din, *self.heads(), self.ld, dout.stride(0),
                                     din.stride(0), self.norm, self.positions, self.inv_freq,
                                     self.spec, grads, accumulate, scratch, st) == 0
        check_status(st)
        assert float(scratch[-1]) == KEEP
        if not in_place:
            assert (din[T:] == KEEP).all() and (din[:, w:] == KEEP).all()
        else:
            assert torch.equal(din[:, w:], self.dout[:, w:])
        return din[:T, :w]

    def check_backward(self):
        T, w, d, H = self.tokens, self.H * self.d, self.d, self.H
        x, qh, kh, eps, centred, gains = self.oracle_args()
        dout = to_f64(self.dout)[:, :w].reshape(T, H, d)
        dx, size, sums = O.qk_norm_backward(x, dout, qh, kh, eps, centred, gains, self.turn)
        # dx: terms as large as the head's largest (pairs mix, means are shared);
        # a centred head loses what its mean takes off
        n, r = O._moments(x, eps, centred)
        lost = 1.0 + (np.abs(x).max(axis=2, keepdims=True) * r if centred else 0.0)
        big = size.max(axis=2, keepdims=True) * lost
        tol = torch.finfo(self.dtype).eps / 2 * np.abs(dx) + F32 * big
        buf = torch.full((4, d), KEEP, device=DEV)
        names = ("q_gain", "k_gain", "q_shift", "k_shift")
        grads = L.make_qk_norm_grads(**dict(zip(names, buf)))
        din = self.backward(grads)
        off = np.abs(to_f64(din).reshape(T, H, d) - dx) / tol
        assert off.max() <= 1, f"dx: {off.max():.3g} of the tolerance"
        got = to_f64(buf)
        worst = float(np.broadcast_to(lost, (T, H, 1)).max())
        tols = []
        for i, (val, mass) in enumerate(s for pair in sums for s in pair):
            if (qh, kh)[i & 1] == 0:
                assert (got[i] == KEEP).all()
                tols.append(np.zeros(d))
                continue
            # a term has the error of its factors, a sum that of its partial sums
            tols.append(F32 * (mass + np.abs(dout).max() * worst) + 2.0 ** -20 * mass.max())
            off = np.abs(got[i] - val) / tols[-1]
            assert off.max() <= 1, f"{names[i]}: {off.max():.3g} of the tolerance"
        # added to what is there, in place, and the same bits
        again = buf.clone()
        grads = L.make_qk_norm_grads(**dict(zip(names, again)))
        assert torch.equal(self.backward(grads, accumulate=1, in_place=True), din)
        used = [i for i in range(4) if (qh, kh)[i & 1]]
        assert torch.equal(again[used], 2 * buf[used])
        # some of them, or none
        one = torch.full((4, d), KEEP, device=DEV)
        assert torch.equal(self.backward(L.make_qk_norm_grads(q_gain=one[0], k_shift=one[3])), din)
        assert torch.equal(one[0], buf[0]) and torch.equal(one[3], buf[3]) and (one[1:3] == KEEP).all()
        assert torch.equal(self.backward(None), din)
        return self


CASES = [
    dict(tokens=1, q_heads=12, k_heads=12, d=64, rot=64),
    dict(tokens=5, q_heads=3, k_heads=1, d=128, rot=128, sections=[24, 20, 20], extra=128),
    dict(tokens=5, q_heads=2, k_heads=2, d=128, rot=128, sections=[24, 20, 20], dealt=True,
         centred=True, extra=128),
    dict(tokens=130, q_heads=5, k_heads=3, d=128, rot=64, sections=[10, 12, 6, 4], adjacent=True,
         dealt=True, extra=64),
    dict(tokens=7, q_heads=4, k_heads=4, d=64, rot=64, adjacent=True, dtype=torch.float32),
    dict(tokens=3, q_heads=2, k_heads=1, d=80, rot=36, sections=[8, 10], extra=3),  # one by one
    dict(tokens=9, q_heads=1, k_heads=0, d=6, rot=2, dtype=torch.float32, extra=1),
    dict(tokens=9, q_heads=0, k_heads=2, d=7, rot=4, centred=True),
    dict(tokens=4, q_heads=2, k_heads=2, d=96, rot=60, sections=[10, 20], adjacent=True, extra=2),
    dict(tokens=33, q_heads=2, k_heads=2, d=256, rot=256, sections=[64, 64], dtype=torch.float32,
         extra=4),
    dict(tokens=33, q_heads=2, k_heads=2, d=256, rot=128, centred=True),
    dict(tokens=20, q_heads=3, k_heads=2, d=255, rot=130, dtype=torch.float32),
    dict(tokens=20, q_heads=3, k_heads=2, d=250, rot=100, adjacent=True),
    dict(tokens=300, q_heads=64, k_heads=8, d=128, rot=128, extra=1024),
    dict(tokens=600, q_heads=7, k_heads=7, d=64, rot=32, sections=[0, 16], centred=True),
    dict(tokens=11, q_heads=3, k_heads=2, d=64, rot=24, adjacent=True),   # vectors that do not pair up
    dict(tokens=6, q_heads=2, k_heads=1, d=72, rot=48),
    dict(tokens=6, q_heads=2, k_heads=1, d=72, rot=64, sections=[20, 12], adjacent=True, dealt=True,
         dtype=torch.float32),
    dict(tokens=50, q_heads=4, k_heads=4, d=128),                          # nothing turns
    dict(tokens=50, q_heads=4, k_heads=0, d=64, gains=False, centred=True, shifts=False),
    dict(tokens=3, q_heads=1, k_heads=1, d=1, centred=False),
    dict(tokens=50, q_heads=2, k_heads=2, d=40, rot=40, gains=False, shifts=True),
]


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    Problem(**case).check_forward()


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    Problem(**case).check_backward()


def test_many_tokens():
    """More items than there are warps, groups of tokens that end unevenly."""
    for p in (Problem(20011, 2, 1, 64, 64, centred=True), Problem(5003, 12, 4, 128, 64)):
        p.x = p.x.clone()
        p.check_forward().check_backward()


def test_a_head_of_zeros():
    p = Problem(4, 2, 2, 64, 64, centred=True)
    p.x[1, :64] = 0
    p.check_forward()
    p.x[2, 64:128] = 2.5  # nothing is left when the mean is off
    p.check_forward()


def test_offsets_past_32_bits():
    tokens, ld = 70000, 32768
    x = torch.zeros(tokens, ld, dtype=torch.bfloat16, device=DEV)
    x[-3:, :256] = torch.randn(3, 256, generator=torch.Generator().manual_seed(8)).bfloat16().to(DEV)
    want = O.qk_norm(to_f64(x[-3:, :256]).reshape(3, 2, 128), 1, 1, 1e-5, False).reshape(3, -1)
    st = status()
    assert L.mc_qk_norm_forward(x, x, tokens, 1, 1, 128, ld, ld, L.make_qk_norm(), status=st) == 0
    check_status(st)
    assert (np.abs(to_f64(x[-3:, :256]) - want) <= 2.0 ** -8 * np.abs(want) + F32 * 4).all()
    assert not x[-3:, 256:].any() and not x[:-3].any()
