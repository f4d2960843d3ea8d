"""The polynomial 2^z of the packed attention (packed_fwd.cuh, exp2_fma2), emulated step by step in
float32: no GPU needed.

* Its constants are those of exp2_poly2, and from 2^-126 on its error has the same bound.
* Below, down to -inf, it is off by 2^-127 at most, and -inf is zero in 16 bits.
* NaN stays a value that is not finite in 16 bits.
"""
import os
import re

import numpy as np
import torch

from fwd_bwd_b200.exp2_fit import DEGREE, coefficients_f32

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = open(os.path.join(ROOT, "fwd_bwd_b200", "csrc", "packed_fwd.cuh")).read()
BODY = SRC[SRC.index("float2 exp2_fma2("):]
BODY = BODY[:BODY.index("\n}")]


def _exp2(z):
    c = np.array([np.float32(dict(re.findall(r"kC(\d) = ([0-9.e+-]+)f", BODY))[str(i)])
                  for i in range(DEGREE + 1)], np.float32)
    assert np.array_equal(c, coefficients_f32())
    low = re.findall(r"fmax_nan\(z\.[xy], (-\d+\.0)f\)", BODY)
    assert len(low) == 2 and low[0] == low[1]
    z = np.asarray(z, np.float32)
    zc = np.maximum(z, np.float32(low[0]))  # NaN passes
    magic = np.float32(12582912.0)
    t = (zc + magic).astype(np.float32)
    f = (zc - (t - magic)).astype(np.float32)
    q = np.full(f.shape, c[-1], np.float32)
    for ck in c[-2::-1]:  # a product of two float32 is exact in float64: one rounding per step
        q = (q.astype(np.float64) * f.astype(np.float64) + np.float64(ck)).astype(np.float32)
    bits = np.where(np.isnan(q), np.uint32(0x7FFFFFFF), q.view(np.uint32))  # the device's NaN
    tb = np.where(np.isnan(t), np.uint32(0x7FFFFFFF), t.view(np.uint32))
    with np.errstate(over="ignore"):
        return (bits + (tb << np.uint32(23))).view(np.float32)


def test_normal_range():
    z = np.linspace(-126.0, 16.0, 2_000_001).astype(np.float32)
    rel = np.abs(_exp2(z).astype(np.float64) / np.exp2(z.astype(np.float64)) - 1.0)
    assert rel.max() < 2.5e-7


def test_below_the_normal_range():
    z = np.concatenate([np.linspace(-130.0, -126.0, 400_001), [-1e3, -1e38, -np.inf]])
    z = z.astype(np.float32)
    off = np.abs(_exp2(z).astype(np.float64) - np.exp2(z.astype(np.float64)))
    assert off.max() <= 2.0 ** -127
    zero = torch.from_numpy(_exp2([-np.inf, -1e3]))
    assert not zero.bfloat16().any() and not zero.half().any()


def test_nan_is_not_finite_in_16_bits():
    x = torch.from_numpy(_exp2([np.nan]))
    assert not torch.isfinite(x.bfloat16()).any() and not torch.isfinite(x.half()).any()
