"""Packed attention where scores are not finite.

By the definition a visible key whose score is NaN or +inf makes its rows NaN (exp(z - max) has no
value), and one whose score is -inf weighs exactly nothing.  Every column of a key tile and of a
query tile is planted in turn, because the kernels treat columns differently (part of the
exponentials are polynomials, the tiles on the causal diagonal are masked).
"""
import math

import pytest
import torch

import packed_ref as R
from fwd_bwd_b200 import ops, packed

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
KINDS = [(64, BF), (64, HF), (128, BF), (128, HF)]


def _inputs(T, hq, hkv, d, dt, seed):
    """q, k, v, do; channel 0 of q is positive, so an infinity there in k gives one of its sign."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, do = (torch.randn((T, h, d), generator=g, device="cuda").to(dt)
                   for h in (hq, hkv, hkv, hq))
    q[..., 0] = q[..., 0].abs() + 0.5
    return q, k, v, do


def _run(q, k, v, do, batch, causal):
    o, lse = packed.attn_fwd(q, k, v, batch, causal)
    dq, dk, dv = packed.attn_bwd(q, k, v, o, lse, do, batch, causal)
    torch.cuda.synchronize()
    assert ops.device_status() == 0
    return o, lse, dq, dk, dv


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [(2, 1), (3, 3)], ids=str)
@pytest.mark.parametrize("d,dt", KINDS)
def test_one_key_of_every_column(d, dt, heads, causal, value):
    """128 sequences of three whole tiles; in sequence s, one channel of key 128 + s is planted."""
    n, S = 384, 128
    q, k, v, do = _inputs(n * S, *heads, d, dt, 80)
    batch = packed.Batch([n] * S)
    clean = _run(q, k, v, do, batch, causal)
    bad = k.clone()
    key = torch.arange(S, device="cuda") + 128
    bad.view(S, n, heads[1], d)[torch.arange(S, device="cuda"), key, :, 0] = value
    o, lse, dq, dk, dv = _run(q, bad, v, do, batch, causal)
    row = torch.arange(n, device="cuda")
    sees = (row >= key[:, None]).flatten() if causal else torch.ones(n * S, dtype=torch.bool,
                                                                     device="cuda")
    assert torch.isnan(o[sees]).all() and not torch.isfinite(lse[:, sees]).any()
    assert torch.equal(o[~sees], clean[0][~sees])
    assert torch.equal(lse[:, ~sees], clean[1][:, ~sees])
    assert torch.isnan(dq[sees]).all()
    # every key is seen by a row that sees the planted one
    assert not torch.isfinite(dv).any() and not torch.isfinite(dk).any()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,dt", KINDS)
def test_one_query_of_every_column(d, dt, causal):
    """A NaN in query 128 + s of sequence s: its own row, and the gradients of the keys it sees."""
    n, S = 384, 128
    q, k, v, do = _inputs(n * S, 2, 1, d, dt, 81)
    batch = packed.Batch([n] * S)
    clean = _run(q, k, v, do, batch, causal)
    bad = q.clone()
    at = torch.arange(S, device="cuda") * n + 128 + torch.arange(S, device="cuda")
    bad[at, :, 3] = math.nan
    o, lse, dq, dk, dv = _run(bad, k, v, do, batch, causal)
    own = torch.zeros(n * S, dtype=torch.bool, device="cuda")
    own[at] = True
    assert torch.isnan(o[own]).all() and torch.isnan(lse[:, own]).all()
    assert torch.isnan(dq[own]).all()
    assert torch.equal(o[~own], clean[0][~own]) and torch.equal(lse[:, ~own], clean[1][:, ~own])
    row = torch.arange(n * S, device="cuda")
    seen = (row <= at.repeat_interleave(n)) if causal else torch.ones_like(own)
    assert not torch.isfinite(dv[seen]).any() and not torch.isfinite(dk[seen]).any()
    # a hidden key's P is exactly zero, and the row's dO is finite
    assert torch.equal(dv[~seen], clean[4][~seen])


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,dt", KINDS)
def test_one_key_where_walks_are_cut_into_parts(d, dt, causal, value):
    n = 4096
    q, k, v, do = _inputs(n, 1, 1, d, dt, 82)
    batch = packed.Batch([n])
    assert packed.fwd_workspace_bytes(q, k, v, batch, causal) > 0
    clean = _run(q, k, v, do, batch, causal)
    for col in range(64):
        key = 1280 + col + 64 * (col % 40)  # every column of a run of 64, over several parts
        bad = k.clone()
        bad[key, 0, 0] = value
        o, lse, dq, dk, dv = _run(q, bad, v, do, batch, causal)
        first = key if causal else 0
        assert torch.isnan(o[first:]).all() and not torch.isfinite(lse[:, first:]).any(), key
        assert torch.equal(o[:first], clean[0][:first]), key
        assert torch.isnan(dq[first:]).all(), key
        assert not torch.isfinite(dv).any() and not torch.isfinite(dk).any(), key


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,dt", KINDS)
def test_scores_of_minus_infinity_weigh_nothing(d, dt, causal):
    """Keys whose scores are -inf, whole tiles of them first and single ones later: the outputs are
    the definition's.  Rows that see no other key have none: NaN, LSE -inf."""
    lengths = [640, 500]
    q, k, v, _ = _inputs(sum(lengths), 2, 1, d, dt, 83)
    k[:300, :, 0] = -math.inf      # of the first sequence
    k[320:640:7, :, 0] = -math.inf
    k[640 + 3:640 + 400:5, :, 0] = -math.inf
    batch = packed.Batch(lengths)
    o, lse = packed.attn_fwd(q, k, v, batch, causal)
    assert ops.device_status() == 0
    ref = R.attention(q, k, v, lengths, causal, d ** -0.5)
    some = torch.ones(sum(lengths), dtype=torch.bool, device="cuda")
    if causal:
        some[:300] = False
    cut = {n: (x[some] if n.startswith("o") else x[:, some]) for n, x in ref.items()
           if n in ("o", "o_tol", "lse", "lse_tol")}
    R.close(o[some], cut, "o")
    R.close(lse[:, some], cut, "lse")
    assert torch.isnan(o[~some]).all()
    assert bool((lse[:, ~some] == -math.inf).all())


@pytest.mark.parametrize("lengths,heads", [([256, 130, 384], (2, 1)), ([4096], (1, 1))], ids=str)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,dt", KINDS)
def test_no_score_but_minus_infinity(d, dt, causal, lengths, heads):
    q, k, v, _ = _inputs(sum(lengths), *heads, d, dt, 84)
    k[..., 0] = -math.inf
    o, lse = packed.attn_fwd(q, k, v, packed.Batch(lengths), causal)
    assert ops.device_status() == 0
    assert torch.isnan(o).all() and bool((lse == -math.inf).all())
