"""Rotary angles of positions beyond 32 bits against turns in exact rational arithmetic."""
import math
from fractions import Fraction

import pytest
import torch

import packed_ref as R
from fwd_bwd_b200 import rope

pytestmark = pytest.mark.gpu

# 2 pi to 60 digits
TWO_PI = Fraction("6.28318530717958647692528676655900576839433879875021164194989")


def _angle(pos, freq):
    """pos * freq modulo a turn, freq the double itself."""
    turns = Fraction(pos) * Fraction(freq) / TWO_PI
    return float((turns - math.floor(turns)) * TWO_PI)


@pytest.mark.parametrize("base", [10000.0, 1e6])
@pytest.mark.parametrize("at", [(1 << 32) + 5, -(1 << 33) - 1, 1 << 40, -(1 << 40) + 3, 1 << 50])
def test_far_positions(at, base):
    T, d, half = 9, 64, 32
    g = torch.Generator(device="cuda").manual_seed(90)
    q, k, dq, dk = (torch.randn((T, h, d), generator=g, device="cuda").half() for h in (2, 1, 2, 1))
    rp = rope.Rope(d, base=base, norm=False)
    pos = [at + 7 * i for i in range(T)]
    angle = torch.tensor([[_angle(p, f) for f in rp.inv_freq] for p in pos], dtype=torch.float64,
                         device="cuda")[:, None]
    at_dev = torch.tensor(pos, device="cuda")
    outs = rope.qk_norm_rope_fwd(q, k, at_dev, rp)
    grads = rope.qk_norm_rope_bwd(q, k, dq, dk, at_dev, rp)
    # the fast sine 2^-21, three roundings of an angle below pi to 2^-24 and the frequency's to
    # 2^-65 turns (of 1.4: the host's quotient has 64 bits); the sums in float32
    off = (2.0 ** -21 + 3 * math.pi * 2.0 ** -24 + 1.4 * 2 * math.pi * abs(at) * 1.01 * 2.0 ** -65
           + 2 * math.pi * 2.0 ** -32 + 4 * R.F32)
    for x, y, sign in ((q, outs[0], 1), (k, outs[1], 1), (dq, grads[0], -1), (dk, grads[1], -1)):
        a, b = x[..., :half].double(), x[..., half:].double()
        c, s = angle.cos(), sign * angle.sin()
        want = torch.cat([a * c - b * s, b * c + a * s], -1)
        tol = off * (a.abs() + b.abs()).repeat(1, 1, 2) + R.unit(x.dtype) * want.abs() * (
            1 + off) + R.tiny(x.dtype)
        R.close(y, {"y": want, "y_tol": tol}, "y")
