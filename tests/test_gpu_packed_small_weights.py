"""Attention rows whose result comes from small weights: one key holds nearly all the weight and
has v = 0, so the others' bits are all that the output shows."""
import math

import pytest
import torch

import packed_ref as R
from fwd_bwd_b200 import ops, packed

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("lengths,heads", [([700], (2, 1)), ([257, 400], (3, 3)), ([4200], (1, 1))],
                         ids=str)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("log2_weight", [13.828125, 16.265625, 20.296875])
@pytest.mark.parametrize("d,dt", [(64, BF), (64, HF), (128, BF), (128, HF)])
def test_weights_below_the_largest(d, dt, log2_weight, causal, lengths, heads):
    """Weights of 2^-20 of the row's largest keep the type's precision, in half precision too (its
    normal numbers end at 2^-14; the probabilities are held times 2^7).  Equal scores, so that
    roundings of the probabilities do not average out."""
    T = sum(lengths)
    g = torch.Generator(device="cuda").manual_seed(95)
    q, k = (torch.zeros((T, h, d), dtype=dt, device="cuda") for h in heads)
    v = (0.5 + torch.rand((T, heads[1], d), generator=g, device="cuda")).to(dt)
    q[..., 0] = 1.0
    # in bf16 that score has fewer bits: its own value counts
    at = 0
    for n in lengths:
        k[at, :, 0] = log2_weight
        v[at] = 0.0
        at += n
    scale = math.log(2.0)
    o, lse = packed.attn_fwd(q, k, v, packed.Batch(lengths), causal, scale)
    torch.cuda.synchronize()
    assert ops.device_status() == 0
    ref = R.attention(q, k, v, lengths, causal, scale)
    # P and the output are each rounded once; scores, exponentials and sums in float32 (2^-17 of
    # the value: scores of 20 to 2^-24, twice, and 4200 summands)
    want, u = ref["o"], R.unit(dt)
    tol = (2 * u + u * u + 2.0 ** -17 + max(lengths) * R.F32) * want.abs() + R.tiny(dt)
    R.close(o, {"o": want, "o_tol": tol}, "o")
    R.close(lse, ref, "lse")
