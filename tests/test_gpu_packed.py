"""Packed grouped-head attention on the GPU against its 64-bit definition.

Every comparison is element by element against a bound computed with the reference (packed_ref):
one rounding of P, dS and each output to the 16-bit type, float32 sums.
"""
import math

import pytest
import torch

import packed_ref as R
from fwd_bwd_b200 import ops, packed

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _inputs(T, hq, hkv, d, dt, layout="fused", seed=0, do_scale=1e-2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if layout == "fused":  # slices of one projection's output, with columns nobody reads
        x = torch.randn((T, hq + 2 * hkv + 1, d), generator=g, device="cuda").to(dt)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]
    elif layout == "heads":  # [H, T, d] storage
        q, k, v = (torch.randn((h, T, d), generator=g, device="cuda").to(dt).transpose(0, 1)
                   for h in (hq, hkv, hkv))
    else:
        q, k, v = (torch.randn((T, h, d), generator=g, device="cuda").to(dt)
                   for h in (hq, hkv, hkv))
    do = (torch.randn((T, hq, d), generator=g, device="cuda") * do_scale).to(dt)
    return q, k, v, do


def _run(q, k, v, do, lengths, causal=True, scale=0.0):
    b = packed.Batch(lengths)
    o, lse = packed.attn_fwd(q, k, v, b, causal, scale)
    dq, dk, dv = packed.attn_bwd(q, k, v, o, lse, do, b, causal, scale)
    torch.cuda.synchronize()
    assert ops.device_status() == 0
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _check(got, q, k, v, do, lengths, causal=True, scale=0.0):
    ref = R.attention(q, k, v, lengths, causal, scale or 1 / math.sqrt(q.shape[2]), do)
    n = sum(lengths)
    for name, x in got.items():
        rows = (slice(None), slice(0, n)) if name == "lse" else slice(0, n)
        part = {name: ref[name][rows], name + "_tol": ref[name + "_tol"][rows]}
        R.close(x[rows], part, name)
    return ref


LENGTHS = [[1], [2], [127], [128], [129], [257], [1, 1, 1], [0, 5, 0, 131, 0],
           [300, 5, 1, 128, 0, 777], [64] * 7, [1500, 3]]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda v: "-".join(map(str, v)))
def test_lengths(lengths, causal):
    q, k, v, do = _inputs(sum(lengths), 2, 1, 128, BF)
    _check(_run(q, k, v, do, lengths, causal), q, k, v, do, lengths, causal)


@pytest.mark.parametrize("layout", ["fused", "heads", "plain"])
@pytest.mark.parametrize("heads", [(1, 1), (2, 1), (3, 1), (6, 2), (5, 5), (16, 2), (12, 4)],
                         ids=str)
@pytest.mark.parametrize("d,dt", [(64, BF), (64, HF), (128, BF), (128, HF)])
def test_heads_types_layouts(heads, d, dt, layout):
    lengths = [200, 1, 333, 0, 130]
    q, k, v, do = _inputs(sum(lengths), *heads, d, dt, layout, seed=heads[0])
    causal = (heads[0] + d // 64) % 2 == 0
    _check(_run(q, k, v, do, lengths, causal), q, k, v, do, lengths, causal)


@pytest.mark.parametrize("dt", [BF, HF])
def test_long_sequence(dt):
    lengths = [4133, 900]
    q, k, v, do = _inputs(sum(lengths), 4, 2, 128, dt, seed=5)
    _check(_run(q, k, v, do, lengths), q, k, v, do, lengths)


@pytest.mark.parametrize("d,dt,heads", [(64, HF, (4, 2)), (128, BF, (4, 2)), (128, BF, (3, 3))])
def test_growing_maximum(d, dt, heads):
    """Scores that rise along the sequence by hundreds: the running maximum is raised, and O
    rescaled, on many key tiles; whole tiles' probabilities vanish."""
    lengths = [1000, 513]
    q, k, v, do = _inputs(sum(lengths), *heads, d, dt, "plain", seed=6)
    ramp = torch.cat([torch.linspace(0.0, 6.0, n, device="cuda") for n in lengths])
    q = (q * 4).contiguous()
    k = (k * (0.2 + ramp[:, None, None])).to(dt)
    for causal in (True, False):
        _check(_run(q, k, v, do, lengths, causal), q, k, v, do, lengths, causal)


@pytest.mark.parametrize("do_scale", [2.0 ** -18, 200.0])
@pytest.mark.parametrize("dt", [BF, HF])
def test_gradient_magnitudes(dt, do_scale):
    """Small and large dO: half precision's dS would vanish or overflow without its factor.  dO
    near half's smallest normal is itself coarse, but it is the input; what the outputs lose to
    their own type's subnormals is in the bound."""
    lengths = [513, 70]
    q, k, v, do = _inputs(sum(lengths), 4, 2, 64, dt, seed=7, do_scale=do_scale)
    _check(_run(q, k, v, do, lengths), q, k, v, do, lengths)


def test_zero_gradient_and_zero_inputs():
    lengths = [200, 31]
    q, k, v, do = _inputs(sum(lengths), 2, 2, 64, HF)
    got = _run(q, k, v, torch.zeros_like(do), lengths)
    for n in ("dq", "dk", "dv"):
        assert not got[n].any(), n
    z = torch.zeros_like(k)
    got = _run(q, z, z, do, lengths)  # uniform attention over zero values
    assert not got["o"].any() and not got["dq"].any()
    _check(got, q, z, z, do, lengths)


@pytest.mark.parametrize("scale", [0.01, 0.5])
def test_softmax_scale(scale):
    lengths = [140, 9]
    q, k, v, do = _inputs(sum(lengths), 2, 1, 64, BF)
    _check(_run(q, k, v, do, lengths, True, scale), q, k, v, do, lengths, True, scale)


@pytest.mark.parametrize("heads", [(2, 1), (1, 1)], ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_sequences_never_touch(causal, heads):
    """NaN and infinity in some sequences and behind the last one: the others' results are bit
    for bit those without them, and the rows behind the last stay as they were."""
    lengths = [130, 77, 300, 1, 255]
    n, extra = sum(lengths), 140
    q, k, v, do = _inputs(n + extra, *heads, 128, HF, "plain", seed=8)
    clean = _run(q, k, v, do, lengths, causal)
    bad = [x.clone() for x in (q, k, v, do)]
    at = 0
    good = torch.zeros(n + extra, dtype=torch.bool, device="cuda")
    for i, m in enumerate(lengths):
        if i % 2 == 0:
            good[at:at + m] = True
        else:
            for j, x in enumerate(bad):
                x[at:at + m] = [math.nan, math.inf, -math.inf, math.nan][(i + j) % 4]
        at += m
    for x in bad:
        x[n:] = math.nan
    b = packed.Batch(lengths)
    o = torch.full_like(q, 7.0)
    lse = torch.full((heads[0], n + extra), 7.0, device="cuda")
    grads = [torch.full_like(x, 7.0) for x in (q, k, v)]
    packed.attn_fwd(*bad[:3], b, causal, o=o, lse=lse)
    packed.attn_bwd(*bad[:3], o, lse, bad[3], b, causal, dq=grads[0], dk=grads[1], dv=grads[2])
    torch.cuda.synchronize()
    assert ops.device_status() == 0
    for name, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse.t(), *grads)):
        want = clean[name].t() if name == "lse" else clean[name]
        assert torch.equal(x[good], want[good]), name
        assert bool((x[n:] == 7.0).all()), name
    for name, x in clean.items():  # new outputs: zero there
        assert not (x[:, n:] if name == "lse" else x[n:]).any(), name


def test_padded_rows_of_new_outputs_are_zero_in_autograd():
    lengths = [100, 20]
    q, k, v, _ = _inputs(150, 2, 1, 64, BF, "plain")
    q, k, v = (x.clone().requires_grad_(True) for x in (q, k, v))
    o = packed.packed_attention(q, k, v, packed.Batch(lengths))
    o.sum().backward()  # the gradient is a broadcast scalar
    for x in (q, k, v):
        assert not x.grad[120:].any() and torch.isfinite(x.grad).all()


def test_autograd_equals_the_calls():
    lengths = [222, 90]
    q, k, v, do = _inputs(sum(lengths), 4, 2, 128, BF, "fused")
    got = _run(q, k, v, do, lengths)
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v)]
    o = packed.packed_attention(*leaves, packed.Batch(lengths))
    o.backward(do)
    assert torch.equal(o, got["o"])
    for x, n in zip(leaves, ("dq", "dk", "dv")):
        assert torch.equal(x.grad, got[n]), n
    # keys and values given once for all heads (a broadcast input): their gradients add up
    k1 = k[:, :1].clone().requires_grad_(True)
    o = packed.packed_attention(q, k1.expand(-1, 2, -1), v, packed.Batch(lengths))
    o.backward(do)
    kk = k[:, :1].expand(-1, 2, -1).contiguous()
    want = _run(q, kk, v, do, lengths)["dk"]
    assert torch.equal(k1.grad, want.sum(1, keepdim=True))


def test_same_bits_every_time():
    lengths = [700, 300, 45]
    q, k, v, do = _inputs(sum(lengths), 8, 2, 128, BF, seed=9)
    first = _run(q, k, v, do, lengths)
    for _ in range(3):
        again = _run(q, k, v, do, lengths)
        for n in first:
            assert torch.equal(first[n], again[n]), n


def test_sequence_alone_equals_sequence_in_a_batch():
    lengths = [129, 300, 64]
    q, k, v, do = _inputs(sum(lengths), 6, 2, 64, BF, seed=10)
    whole = _run(q, k, v, do, lengths)
    at = 0
    for n in lengths:
        r = slice(at, at + n)
        one = _run(q[r], k[r], v[r], do[r], [n])
        for name in ("o", "dq", "dk", "dv"):
            assert torch.equal(whole[name][r], one[name]), (n, name)
        assert torch.equal(whole["lse"][:, r], one["lse"])
        at += n


def test_strided_outputs():
    lengths = [150, 61]
    T = sum(lengths)
    q, k, v, do = _inputs(T, 4, 2, 64, BF)
    want = _run(q, k, v, do, lengths)
    b = packed.Batch(lengths)
    fused = torch.zeros((T, 4 + 2 * 2, 64), dtype=BF, device="cuda")
    o = torch.zeros((4, T, 64), dtype=BF, device="cuda").transpose(0, 1)
    _, lse = packed.attn_fwd(q, k, v, b, o=o)
    packed.attn_bwd(q, k, v, o, lse, do, b, dq=fused[:, :4], dk=fused[:, 4:6], dv=fused[:, 6:])
    assert torch.equal(o, want["o"])
    assert torch.equal(fused, torch.cat([want["dq"], want["dk"], want["dv"]], 1))


def test_side_stream_and_graph():
    lengths = [333, 128, 7]
    q, k, v, do = _inputs(sum(lengths), 4, 2, 64, HF, "plain", seed=11)
    b = packed.Batch(lengths)
    want = _run(q, k, v, do, lengths)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, lse = packed.attn_fwd(q, k, v, b)
        grads = packed.attn_bwd(q, k, v, o, lse, do, b)
    side.synchronize()
    for n, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
        assert torch.equal(x, want[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = packed.attn_fwd(q, k, v, b)
        grads = packed.attn_bwd(q, k, v, o, lse, do, b)
    for seed in (11, 12, 13):
        for x, y in zip((q, k, v, do), _inputs(sum(lengths), 4, 2, 64, HF, "plain", seed=seed)):
            x.copy_(y)
        for x in (o, lse, *grads):
            x.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert ops.device_status() == 0
        want = _run(q, k, v, do, lengths)
        for n, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
            assert torch.equal(x, want[n]), (seed, n)


def test_backward_captured_beside_a_live_eager_graph():
    lengths = [90, 40]
    q, k, v, do = _inputs(sum(lengths), 2, 1, 64, BF, "plain")
    b = packed.Batch(lengths)
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v)]
    eager = packed.packed_attention(*leaves, b)  # its graph stays alive over the capture
    graph = torch.cuda.CUDAGraph()
    copies = [x.detach().clone().requires_grad_(True) for x in leaves]
    with torch.cuda.graph(graph):
        o = packed.packed_attention(*copies, b)
        grads = torch.autograd.grad(o, copies, do)
    graph.replay()
    eager.backward(do)
    torch.cuda.synchronize()
    for x, g in zip(leaves, grads):
        assert torch.equal(x.grad, g)


def test_rows_past_2_31_elements():
    """Offsets beyond 32 bits: the last sequence's rows lie past 2^32 bytes and 2^31 elements."""
    hq, d = 2, 64
    stride = 1 << 21  # elements from token to token
    T = 1100
    store = torch.empty((T, stride), dtype=BF, device="cuda")
    small = _inputs(T, hq, 1, d, BF, "plain", seed=14)
    q = store[:, :hq * d].unflatten(1, (hq, d))
    k = store[:, 1024:1024 + d].unflatten(1, (1, d))
    v = store[:, 2048:2048 + d].unflatten(1, (1, d))
    for x, y in zip((q, k, v), small):
        x.copy_(y)
    lengths = [1000, 100]
    want = _run(*small, lengths)
    o = store[:, 4096:4096 + hq * d].unflatten(1, (hq, d))
    b = packed.Batch(lengths)
    _, lse = packed.attn_fwd(q, k, v, b, o=o)
    dq, dk, dv = packed.attn_bwd(q, k, v, o, lse, small[3], b)
    for n, x in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(x, want[n]), n


def test_refusals_on_device_tensors():
    q, k, v, do = _inputs(10, 4, 2, 64, BF, "plain")
    b = packed.Batch([10])
    ok = lambda **kw: packed.attn_fwd(**{**dict(q=q, k=k, v=v, batch=b), **kw})  # noqa: E731
    o, lse = ok()
    cases = [dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:, :3]), dict(k=k[:9]), dict(v=v[:, :1]),
             dict(q=q[..., :32]), dict(v=v.to(HF)), dict(batch=packed.Batch([11])),
             dict(batch=packed.Batch([10], device="cpu")), dict(q=q[0]),
             dict(k=k[:, :1].expand(-1, 2, -1)), dict(o=o[:, :2]), dict(lse=lse.t()),
             dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))]
    for kw in cases:
        with pytest.raises((ValueError, RuntimeError)):
            ok(**kw)
    overlap = torch.zeros((10, 64 * 2), dtype=BF, device="cuda").as_strided((10, 4, 64), (64, 64, 1))
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        ok(o=overlap)
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        ok(softmax_scale=math.inf)
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        packed.attn_bwd(q, k, v, o, lse, do, b,
                        workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert packed.workspace_bytes(q, k, v, b) >= 4 * 10 * 4


def test_only_empty_sequences():
    q, k, v, do = _inputs(5, 2, 1, 64, BF, "plain")
    got = _run(q, k, v, do, [0, 0])
    assert not any(x.any() for x in got.values())


@pytest.mark.parametrize("d,heads", [(64, (8, 8)), (64, (9, 3)), (128, (8, 8)), (128, (12, 4))],
                         ids=str)
def test_many_tiles_on_a_full_device(d, heads):
    """More tiles than the device holds at once, many keys per tile: every pipeline's buffers turn
    over many times while other CTAs share the SMs."""
    lengths = [2048, 1900, 1337, 700, 640, 511]
    q, k, v, do = _inputs(sum(lengths), *heads, d, BF, seed=21)
    for causal in (True, False):
        _check(_run(q, k, v, do, lengths, causal), q, k, v, do, lengths, causal)


def test_repeated_launches_finish():
    """Back-to-back launches of every kernel on a full device: no bounded wait runs out."""
    for d in (64, 128):
        lengths = [1024] * 12
        q, k, v, do = _inputs(sum(lengths), 16, 8, d, BF, seed=22)
        b = packed.Batch(lengths)
        want = None
        for _ in range(30):
            o, lse = packed.attn_fwd(q, k, v, b)
            grads = packed.attn_bwd(q, k, v, o, lse, do, b)
            if want is None:
                want = (o, lse, *grads)
        torch.cuda.synchronize()
        assert ops.device_status() == 0
        for x, y in zip(want, (o, lse, *grads)):
            assert torch.equal(x, y)


def test_batch_of_another_layer_and_two_graphs():
    """One Batch under two captured graphs with workspaces of their own, replayed in turn."""
    lengths = [260, 90]
    b = packed.Batch(lengths)
    sets, graphs = [], []
    for seed, (hq, hkv, d, dt) in enumerate([(4, 2, 64, HF), (3, 3, 128, BF)]):
        q, k, v, do = _inputs(sum(lengths), hq, hkv, d, dt, "plain", seed=30 + seed)
        ws = torch.empty(packed.workspace_bytes(q, k, v, b), dtype=torch.uint8, device="cuda")
        o, lse = packed.attn_fwd(q, k, v, b)
        packed.attn_bwd(q, k, v, o, lse, do, b, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            packed.attn_fwd(q, k, v, b, o=o, lse=lse)
            grads = packed.attn_bwd(q, k, v, o, lse, do, b, workspace=ws)
        sets.append((q, k, v, do, o, lse, grads))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert ops.device_status() == 0
    for q, k, v, do, o, lse, grads in sets:
        want = _run(q, k, v, do, lengths)
        for n, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
            assert torch.equal(x, want[n]), n


def test_threads_and_streams_at_once():
    """Two host threads on streams of their own, each with its own tensors."""
    import threading

    lengths = [400, 128, 33]
    b = packed.Batch(lengths)
    inputs = [_inputs(sum(lengths), 4, 2, 64 * (1 + i % 2), BF, "plain", seed=40 + i)
              for i in range(2)]
    want = [_run(*x, lengths) for x in inputs]
    got, errors = [None, None], []
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                q, k, v, do = inputs[i]
                for _ in range(5):
                    o, lse = packed.attn_fwd(q, k, v, b)
                    grads = packed.attn_bwd(q, k, v, o, lse, do, b)
                torch.cuda.current_stream().synchronize()
                got[i] = (o, lse, *grads)
        except Exception as e:  # noqa: BLE001 - reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert ops.device_status() == 0
    for i in range(2):
        for n, x in zip(("o", "lse", "dq", "dk", "dv"), got[i]):
            assert torch.equal(x, want[i][n]), (i, n)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
def test_single_keys_have_no_score_gradient(d, dt):
    """Sequences of one token: P = 1, so dQ and dK vanish (to float32 rounding of dP) and dV = dO."""
    lengths = [1] * 50
    q, k, v, do = _inputs(50, 2, 1, d, dt, "plain", seed=50, do_scale=1.0)
    got = _run(q, k, v, do, lengths)
    R.close(got["dv"], R.attention(q, k, v, lengths, True, d ** -0.5, do), "dv")
    size = (do.double().abs()[:, :, None] * v.double().abs()[:, None]).sum(-1).max()
    # dS = P dP - P (P dP) with P = exp2 of a rounding error: |dS| <= 2^-18 |dO| |v|
    for n, other in (("dq", k), ("dk", q)):
        assert float(got[n].double().abs().max()) <= float(
            2.0 ** -18 * size * d ** -0.5 * other.double().abs().max() * 2 + R.tiny(dt)), n


def test_batch_freed_while_another_stream_reads_it():
    """A plan made on one stream, read on another, and dropped at once: its memory is not given to
    new tensors of the first stream while the kernels run."""
    lengths = [1024] * 8
    q, k, v, do = _inputs(sum(lengths), 8, 2, 128, BF, "plain", seed=60)
    want = _run(q, k, v, do, lengths)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            b = packed.Batch(lengths)
        o, lse = packed.attn_fwd(q, k, v, b)
        grads = packed.attn_bwd(q, k, v, o, lse, do, b)
        size = b.plan.numel()
        del b
        with torch.cuda.stream(side):
            junk = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        assert ops.device_status() == 0 and junk
        for n, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
            assert torch.equal(x, want[n]), n


@pytest.mark.parametrize("heads,lengths", [((8, 1), [1500, 40]), ((16, 2), [3000]), ((6, 1), [257, 0, 1024]),
                                           ((1, 1), [4100])], ids=str)
@pytest.mark.parametrize("d,dt", [(64, HF), (128, BF)])
def test_few_key_heads(heads, lengths, d, dt):
    """Few key tiles with long walks: dK and dV are made in parts and joined."""
    q, k, v, do = _inputs(sum(lengths) + 3, *heads, d, dt, "fused", seed=70)
    for causal in (True, False):
        got = _run(q, k, v, do, lengths, causal)
        _check(got, q, k, v, do, lengths, causal)
        again = _run(q, k, v, do, lengths, causal)
        for n in ("dk", "dv"):
            assert torch.equal(got[n], again[n])
            assert not got[n][sum(lengths):].any()


@pytest.mark.parametrize("d", [64, 128])
def test_parts_keep_sequences_apart_and_nan_within(d):
    """Walks cut into parts: another sequence's NaN stays there, its own reaches the rows that see
    it (whole parts of NaN scores too), and rows of earlier tiles stay finite."""
    lengths = [300, 4096]
    q, k, v, do = _inputs(sum(lengths), 1, 1, d, BF, "plain", seed=71)
    b = packed.Batch(lengths)
    assert packed.fwd_workspace_bytes(q, k, v, b) > 0
    clean = _run(q, k, v, do, lengths)
    bad = k.clone()
    bad[:300] = math.nan
    got = _run(q, bad, v, do, lengths)
    for n, x in got.items():
        rows = (slice(None), slice(300, None)) if n == "lse" else slice(300, None)
        assert torch.equal(x[rows], clean[n][rows]), n
    bad = k.clone()
    bad[300 + 1024:300 + 2304] = math.nan
    o, lse = packed.attn_fwd(q, bad, v, b)
    assert torch.isnan(o[300 + 1024:]).all() and torch.isnan(lse[:, 300 + 1024:]).all()
    assert torch.equal(o[:300 + 1024], clean["o"][:300 + 1024])


def test_workspace_refusals_of_the_forward():
    q, k, v, _ = _inputs(4096, 1, 1, 64, BF, "plain")
    b = packed.Batch([4096])
    n = packed.fwd_workspace_bytes(q, k, v, b)
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        packed.attn_fwd(q, k, v, b, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        packed.attn_fwd(q, k, v, b, workspace=torch.empty(n, dtype=torch.uint8))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert torch.equal(packed.attn_fwd(q, k, v, b, workspace=ws)[0], packed.attn_fwd(q, k, v, b)[0])


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (3, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_later_values_that_are_not_finite(d, Hq, Hkv):
    """Of a hidden key: its k reaches no earlier row, its v none of the tiles before its own (tiles
    of 128 from the sequence's end: 500 tokens start theirs at -12, 116, 244, 372)."""
    q, k, v, _ = _inputs(500, Hq, Hkv, d, BF, "plain", seed=72)
    b = packed.Batch([500])
    o, lse = packed.attn_fwd(q, k, v, b)
    for value in (math.nan, math.inf):
        bad = k.clone()
        bad[300] = value
        o1, lse1 = packed.attn_fwd(q, bad, v, b)
        assert torch.equal(o1[:300], o[:300]) and torch.equal(lse1[:, :300], lse[:, :300])
        assert torch.isnan(o1[300:]).any(-1).any()
        bad = v.clone()
        bad[300] = value
        o2, lse2 = packed.attn_fwd(q, k, bad, b)
        assert torch.equal(o2[:244], o[:244]) and torch.equal(lse2, lse)
        assert not torch.isfinite(o2[300:]).any()
