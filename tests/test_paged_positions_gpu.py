"""Rotation at far positions and small bases, in fp32, against angles taken from 60-digit arithmetic.

A pair (a, b) turns to (a c - b s, b c + a s). c and s are off by
  2 pi 2^-32             the phase is kept to 2^-32 turn
  2 pi |t| 2^-58.6       frequencies: a factor of at most 2^-2.6 turns, 2 roundings of 2^-64 a step, 128 steps at most
  2.4 2^-24              the angle of at most pi / 4 from the phase: two roundings and a rounded constant
  2^-25                  the Taylor remainder
  2 2^-24                their evaluation,
less than 2^-21.5 together at every int32 position, and the products and their sum are rounded by 2 2^-24 of
|a| + |b|: with the output's own rounding less than 2^-21 (|a| + |b|)."""
from decimal import Decimal, getcontext

import pytest
import torch

pytestmark = pytest.mark.gpu

POSITIONS = [0, 1, -1, 32767, 131071, 2 ** 20 + 3, 2 ** 30 + 12345, 2 ** 31 - 1, -2 ** 31]


def _turned(q, theta, rot):
    """The rotation in 64 bits, with every angle reduced to less than a turn in 60 digits."""
    getcontext().prec = 60
    turn = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    step = (Decimal(theta).ln() * -2 / rot).exp() if theta != 1 else Decimal(1)
    freq = [step ** i for i in range(rot // 2)]
    a = torch.tensor([[float(t * f % turn) for f in freq] for t in POSITIONS], dtype=torch.float64)[:, None]
    x, h, out = q.double().cpu(), rot // 2, q.double().cpu().clone()
    out[..., :h] = x[..., :h] * a.cos() - x[..., h:rot] * a.sin()
    out[..., h:rot] = x[..., h:rot] * a.cos() + x[..., :h] * a.sin()
    return out


@pytest.mark.parametrize("theta", [1.0, 1.25, 2.0, 1e4, 1e6, 2.0 ** 126])
@pytest.mark.parametrize("d,rot", [(256, 256), (128, 64), (64, 16)])
def test_rotation_at_far_positions(cuda_lib, theta, d, rot):
    qsa = cuda_lib
    gen = torch.Generator().manual_seed(d)
    q = torch.randn(len(POSITIONS), 2, d, generator=gen).cuda()
    cfg = qsa.make_config(2, 1, d, 4, 64, 64, 4, "fp32")
    nr = qsa.make_norm_rope(rope_theta=theta, rotary_dim=rot)
    out = torch.empty_like(q)
    qsa.qsa_norm_rope(cfg, nr, torch.tensor(POSITIONS, dtype=torch.int32, device="cuda"), q, None, out, None)
    want, x = _turned(q, theta, rot), q.double().cpu().abs()
    pair = torch.zeros_like(x)
    pair[..., : rot // 2] = pair[..., rot // 2: rot] = x[..., : rot // 2] + x[..., rot // 2: rot]
    over = (out.double().cpu() - want).abs() - 2.0 ** -21 * pair
    assert over.max() <= 0, f"worst {float(over.max()):.3e} at {over.argmax()}"
    assert torch.equal(out[..., rot:], q[..., rot:])
