"""Half precision's factor of dS, which comes from the largest |dO| and |v| of a sequence: values
that are not finite say nothing about the rows that do not see them."""
import math

import pytest
import torch

from fwd_bwd_b200 import ops, packed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_do_not_see_the_value_keep_their_gradient(d, value):
    """Small dO, whose dS would vanish without the factor; NaN or infinity in a late v or dO leaves
    dq of the tiles before it as it was, bit for bit."""
    n, hq, hkv = 640, 4, 2
    g = torch.Generator(device="cuda").manual_seed(97)
    q, k, v, do = (torch.randn((n, h, d), generator=g, device="cuda") for h in (hq, hkv, hkv, hq))
    do *= 2.0 ** -14
    v[600] *= 0.01  # not the largest, so that the factor is the same without it
    do[600] *= 0.01
    q, k, v, do = (x.half() for x in (q, k, v, do))
    batch = packed.Batch([n])
    o, lse = packed.attn_fwd(q, k, v, batch)
    want = packed.attn_bwd(q, k, v, o, lse, do, batch)
    assert want[0][1:].any(-1).all()
    bad = v.clone()
    bad[600] = value
    o1, lse1 = packed.attn_fwd(q, k, bad, batch)
    dq, _, dv = packed.attn_bwd(q, k, bad, o1, lse1, do, batch)
    assert torch.equal(dq[:512], want[0][:512])
    assert not torch.isfinite(dq[600:]).any()
    assert torch.equal(dv, want[2])  # P^T dO has no v
    bad = do.clone()
    bad[600] = value
    dq, dk, _ = packed.attn_bwd(q, k, v, o, lse, bad, batch)
    assert torch.equal(dq[:600], want[0][:600]) and torch.equal(dq[601:], want[0][601:])
    assert not torch.isfinite(dq[600]).any() and not torch.isfinite(dk[:600]).any()
    assert ops.device_status() == 0
