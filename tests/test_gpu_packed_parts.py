"""Walks that are cut into parts: the pairs of head size and type that other tests leave out, other
streams and captured graphs."""
import math

import pytest
import torch

import packed_ref as R
from fwd_bwd_b200 import ops, packed

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _inputs(T, hq, hkv, d, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, do = (torch.randn((T, h, d), generator=g, device="cuda").to(dt)
                   for h in (hq, hkv, hkv, hq))
    return q, k, v, (do * 1e-2)


def _run(q, k, v, do, batch, causal=True):
    o, lse = packed.attn_fwd(q, k, v, batch, causal)
    dq, dk, dv = packed.attn_bwd(q, k, v, o, lse, do, batch, causal)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


@pytest.mark.parametrize("heads,lengths", [((8, 1), [1500, 40]), ((2, 2), [2500, 1, 300]),
                                           ((1, 1), [4100])], ids=str)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,dt", [(64, BF), (128, HF)])
def test_against_the_definition(d, dt, causal, heads, lengths):
    x = _inputs(sum(lengths), *heads, d, dt, 100)
    batch = packed.Batch(lengths)
    rows = packed.workspace_bytes(*x[:3], batch, causal)
    assert rows > 8 * sum(lengths) * heads[0] + 256 * len(lengths)  # more than D and the norms
    got = _run(*x, batch, causal)
    torch.cuda.synchronize()
    assert ops.device_status() == 0
    ref = R.attention(*x[:3], lengths, causal, 1 / math.sqrt(d), x[3])
    for name, y in got.items():
        R.close(y, ref, name)


@pytest.mark.parametrize("d,dt", [(64, HF), (128, BF)])
def test_other_stream_and_graph(d, dt):
    lengths = [3000, 200]
    batch = packed.Batch(lengths)
    x = _inputs(sum(lengths), 2, 1, d, dt, 101)
    assert packed.fwd_workspace_bytes(*x[:3], batch) > 0
    want = _run(*x, batch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _run(*x, batch)
    side.synchronize()
    for name in want:
        assert torch.equal(got[name], want[name]), name
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _run(*x, batch)
    for seed in (101, 102):
        for a, b in zip(x, _inputs(sum(lengths), 2, 1, d, dt, seed)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert ops.device_status() == 0
        want = _run(*x, batch)
        for name in want:
            assert torch.equal(got[name], want[name]), (seed, name)
