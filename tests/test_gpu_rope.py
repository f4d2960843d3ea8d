"""QK-norm with rotary positions on the GPU against its 64-bit definition, and the layer that
uses it before packed and quantized attention."""
import math

import pytest
import torch

import packed_ref as R
from fwd_bwd_b200 import ops, packed, rope

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _case(T, hq, hkv, d, dt, seed=0, layout="fused"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if layout == "fused":
        x = torch.randn((T, hq + 2 * hkv, d), generator=g, device="cuda").to(dt)
        q, k = x[:, :hq], x[:, hq:hq + hkv]
    else:
        q, k = (torch.randn((h, T, d), generator=g, device="cuda").to(dt).transpose(0, 1)
                for h in (hq, hkv))
    dq, dk = (torch.randn((T, h, d), generator=g, device="cuda").to(dt) for h in (hq, hkv))
    gains = [0.5 + torch.rand(d, generator=g, device="cuda") for _ in range(2)]
    return q, k, dq, dk, gains


def _check(q, k, dy, dyk, gains, pos, rp):
    """Forward and backward against the reference; pos [axes, T]."""
    gq, gk = gains
    p = pos[0] if rp.axes == 1 else (pos if rp.axes else None)
    y, yk = rope.qk_norm_rope_fwd(q, k, p, rp, gq, gk)
    dq, dk, dgq, dgk = rope.qk_norm_rope_bwd(q, k, dy, dyk, p, rp, gq, gk)
    for x, gain, up, out, dx, dg in ((q, gq, dy, y, dq, dgq), (k, gk, dyk, yk, dk, dgk)):
        ref = R.rope(x, gain, pos, rp.inv_freq, rp.sections, rp.interleaved, rp.norm, rp.eps, up)
        R.close(out, ref, "y")
        R.close(dx, ref, "dx")
        if rp.norm:
            R.close(dg, ref, "dgain")
        else:
            assert dg is None
    return y, yk


@pytest.mark.parametrize("d,dt", [(64, BF), (64, HF), (128, BF), (128, HF)])
@pytest.mark.parametrize("T,hq,hkv", [(1, 1, 1), (1, 16, 4), (3, 5, 2), (130, 32, 8), (1001, 7, 7),
                                      (4097, 2, 1)])
def test_sizes_and_types(T, hq, hkv, d, dt):
    q, k, dy, dyk, gains = _case(T, hq, hkv, d, dt, T, "fused" if T % 2 else "heads")
    pos = torch.arange(T, device="cuda")[None]
    _check(q, k, dy, dyk, gains, pos, rope.Rope(d))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary,sections", [(0, None), (16, None), (48, None), (64, [10, 12, 10]),
                                             (128, [16, 24, 24]), (112, [1, 2, 50, 3])])
@pytest.mark.parametrize("norm", [True, False])
def test_partial_rotation_axes_and_pairs(rotary, sections, interleaved, norm):
    T = 77
    q, k, dy, dyk, gains = _case(T, 3, 2, 128, BF, 1)
    rp = rope.Rope(128, rotary_dim=rotary, sections=sections, interleaved=interleaved, norm=norm)
    pos = torch.randint(0, 5000, (len(rp.sections), T), device="cuda", dtype=torch.int32)
    _check(q, k, dy, dyk, gains if norm else [None, None], pos, rp)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("at", [-(1 << 31), -70000, (1 << 20) + 3, (1 << 31) - 100])
def test_far_and_negative_positions(at, dtype):
    q, k, dy, dyk, gains = _case(64, 2, 1, 64, HF, 2)
    pos = (torch.arange(64, device="cuda") + at).to(dtype)[None]
    _check(q, k, dy, dyk, gains, pos, rope.Rope(64, base=1e6))


def test_far_position_is_the_rotation_of_a_whole_turn():
    """A frequency of one turn in 64 positions: positions 2^40 turns apart give the same bits."""
    rp = rope.Rope(64, inv_freq=[2 * math.pi / 64] * 32, norm=False)
    q, k, *_ = _case(8, 1, 1, 64, BF, 3)
    pos = torch.arange(8, device="cuda")
    a = rope.qk_norm_rope_fwd(q, k, pos, rp)
    b = rope.qk_norm_rope_fwd(q, k, pos + 64 * 5, rp)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_values_of_every_size():
    """Rows of zeros, tiny and large values: the norm's epsilon and range."""
    q, k, dy, dyk, gains = _case(12, 2, 1, 128, BF, 4)
    scale = torch.tensor([0, 1e-30, 1e-12, 1e-6, 1e-3, 1, 10, 1e3, 1e6, 1e12, 1e15, 1e18],
                         device="cuda")[:, None, None]
    q, k = (q.float() * scale).to(BF), (k.float() * scale).to(BF)
    pos = torch.arange(12, device="cuda")[None]
    y, yk = _check(q, k, dy, dyk, gains, pos, rope.Rope(128))
    assert not y[0].any() and not yk[0].any()


def test_rows_are_independent():
    q, k, dy, dyk, gains = _case(40, 3, 2, 64, HF, 5, "heads")
    rp = rope.Rope(64, rotary_dim=32, norm=False)
    pos = torch.arange(40, device="cuda")
    want = rope.qk_norm_rope_fwd(q, k, pos, rp)
    bad = q.clone()
    bad[7, 1] = math.nan
    bad[9, 0] = math.inf
    got = rope.qk_norm_rope_fwd(bad, k, pos, rp)
    same = torch.ones((40, 3), dtype=torch.bool, device="cuda")
    same[7, 1] = same[9, 0] = False
    assert torch.equal(got[0][same], want[0][same]) and torch.equal(got[1], want[1])
    # the channels behind the rotated ones pass through
    assert bool(torch.isinf(got[0][9, 0, 32:]).all())


def test_batched_layout_and_shared_positions():
    B, N, hq, hkv, d = 3, 50, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(6)
    q = torch.randn((B, hq, N, d), generator=g, device="cuda").to(BF)
    k = torch.randn((B, hkv, N, d), generator=g, device="cuda").to(BF)
    rp = rope.Rope(d, sections=[16, 16])
    pos = torch.randint(0, 900, (2, N), generator=g, device="cuda")
    y, yk = rope.qk_norm_rope_fwd(q, k, pos, rp)
    each = pos[:, None].expand(2, B, N).contiguous()
    y2, yk2 = rope.qk_norm_rope_fwd(q, k, each, rp)
    assert torch.equal(y, y2) and torch.equal(yk, yk2)
    own = each + 100 * torch.arange(B, device="cuda")[None, :, None]
    y3, yk3 = rope.qk_norm_rope_fwd(q, k, own, rp)
    for b in range(B):  # the same as packed rows of one entry
        for pp, yy, yyk in ((pos, y, yk), (own[:, b].contiguous(), y3, yk3)):
            p, pk = rope.qk_norm_rope_fwd(q[b].transpose(0, 1), k[b].transpose(0, 1), pp, rp)
            assert torch.equal(yy[b].transpose(0, 1), p) and torch.equal(yyk[b].transpose(0, 1), pk)


def test_same_bits_streams_and_graph():
    q, k, dy, dyk, gains = _case(3000, 8, 2, 128, BF, 7)
    rp = rope.Rope(128)
    pos = torch.arange(3000, device="cuda")

    def run():
        y = rope.qk_norm_rope_fwd(q, k, pos, rp, *gains)
        return (*y, *rope.qk_norm_rope_bwd(q, k, dy, dyk, pos, rp, *gains))

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for x in captured:
        x.fill_(math.nan)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, captured))


def test_autograd_of_a_layer():
    """Norm, rotation and packed attention in a chain: every stage against its reference on the
    inputs that it got, and autograd equal to the calls."""
    lengths = [200, 1, 131]
    T, hq, hkv, d = sum(lengths), 4, 2, 64
    q, k, _, _, gains = _case(T, hq, hkv, d, BF, 8)
    v = torch.randn((T, hkv, d), device="cuda").to(BF)
    do = (torch.randn((T, hq, d), device="cuda") * 1e-2).to(BF)
    batch = packed.Batch(lengths)
    pos, rp = batch.positions(), rope.Rope(d)
    y, yk = rope.qk_norm_rope_fwd(q, k, pos, rp, *gains)
    o, lse = packed.attn_fwd(y, yk, v, batch)
    dy, dyk, dv = packed.attn_bwd(y, yk, v, o, lse, do, batch)
    dq, dk, dgq, dgk = rope.qk_norm_rope_bwd(q, k, dy, dyk, pos, rp, *gains)
    ref = R.attention(y, yk, v, lengths, True, d ** -0.5, do)
    for name, x in (("o", o), ("lse", lse), ("dq", dy), ("dk", dyk), ("dv", dv)):
        R.close(x, ref, name)
    for x, gain, up, out, dx, dg in ((q, gains[0], dy, y, dq, dgq), (k, gains[1], dyk, yk, dk, dgk)):
        r = R.rope(x, gain, pos[None], rp.inv_freq, rp.sections, False, True, rp.eps, up)
        R.close(out, r, "y")
        R.close(dx, r, "dx")
        R.close(dg, r, "dgain")
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v, gains[0])]
    gk = gains[1].to(BF).requires_grad_(True)  # a gain in the tensors' type
    a, b = rope.qk_norm_rope(leaves[0], leaves[1], pos, rp, leaves[3], gk)
    assert torch.equal(a, y)
    out = packed.packed_attention(a, b, leaves[2], batch)
    out.backward(do)
    assert gk.grad.dtype == BF and torch.isfinite(gk.grad).all()
    # with k's gain rounded to bf16 the chain differs; with the same gains it is the calls' bits
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v, *gains)]
    a, b = rope.qk_norm_rope(leaves[0], leaves[1], pos, rp, leaves[3], leaves[4])
    packed.packed_attention(a, b, leaves[2], batch).backward(do)
    for x, want in zip(leaves, (dq, dk, dv, dgq, dgk)):
        assert torch.equal(x.grad, want)


def test_before_quantized_attention():
    """[B, H, N, d] q and k, rotated, into the INT8 attention (which then skips its own norm)."""
    B, H, N, d = 2, 2, 256, 64
    g = torch.Generator(device="cuda").manual_seed(9)
    q, k, v, do = (torch.randn((B, H, N, d), generator=g, device="cuda").to(BF) for _ in range(4))
    pos, rp = torch.arange(N, device="cuda"), rope.Rope(d)
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v)]
    y, yk = rope.qk_norm_rope(leaves[0], leaves[1], pos, rp)
    o = ops.sage_attention(y, yk, leaves[2], qknorm=False)
    o.backward(do)
    assert ops.device_status() == 0
    cfg = ops.Config(qknorm=False)
    y2, yk2 = rope.qk_norm_rope_fwd(q, k, pos, rp)
    qb = ops.quant_prologue(y2, yk2, v, cfg)
    o2, lse = ops.attn_fwd(qb, y2, cfg)
    assert torch.equal(o, o2)
    # the same rotated q and k through 16-bit attention: the INT8 path is within its 0.5% cosine
    rows = lambda x: x.transpose(1, 2).reshape(B * N, H, d)  # noqa: E731
    o16, _ = packed.attn_fwd(rows(y2), rows(yk2), rows(v), packed.Batch([N] * B))
    a, b = rows(o2).double().flatten(), o16.double().flatten()
    assert float(a @ b / (a.norm() * b.norm())) >= 0.995
    for x in leaves:
        assert torch.isfinite(x.grad).all() and x.grad.any()


def test_refusals_on_device_tensors():
    q, k, dy, dyk, gains = _case(10, 2, 1, 64, BF)
    pos, rp = torch.arange(10, device="cuda"), rope.Rope(64)
    ok = lambda **kw: rope.qk_norm_rope_fwd(**{**dict(  # noqa: E731
        q=q, k=k, positions=pos, rope=rp, gain_q=gains[0], gain_k=gains[1]), **kw})
    ok()
    for kw in (dict(q=q.float()), dict(q=q.cpu()), dict(k=k[:9]), dict(k=k.to(HF)),
               dict(positions=None), dict(positions=pos.float()), dict(positions=pos[:9]),
               dict(positions=pos.cpu()), dict(positions=pos[None].expand(2, 10)),
               dict(gain_q=gains[0].half()), dict(gain_k=gains[1][:32]),
               dict(gain_q=gains[0].cpu()), dict(rope=rope.Rope(128)),
               dict(rope=rope.Rope(64, norm=False)), dict(q=q[0]), dict(q_out=q[:5]),
               dict(k=k[:, :1].expand(-1, 3, -1)), dict(rope=rope.Rope(64, sections=[16, 16]))):
        with pytest.raises((ValueError, RuntimeError)):
            ok(**kw)
    with pytest.raises(ValueError):
        rope.qk_norm_rope_bwd(q, k, dy[:5], dyk, pos, rp, *gains)
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        rope.qk_norm_rope_bwd(q, k, dy, dyk, pos, rp, *gains,
                              workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_no_tokens():
    q, k, dy, dyk, gains = _case(0, 2, 1, 64, BF, layout="heads")
    pos, rp = torch.arange(0, device="cuda"), rope.Rope(64)
    y, yk = rope.qk_norm_rope_fwd(q, k, pos, rp, *gains)
    assert y.shape == (0, 2, 64) and yk.shape == (0, 1, 64)
    *_, dgq, dgk = rope.qk_norm_rope_bwd(q, k, dy, dyk, pos, rp, *gains)
    assert not dgq.any() and not dgk.any()


@pytest.mark.parametrize("d,hq,hkv,inter", [(64, 5, 3, False), (128, 6, 1, True)])
def test_many_units_per_block(d, hq, hkv, inter):
    """Every block walks many tiles of tokens, with odd numbers of heads."""
    T = 30011
    q, k, dy, dyk, gains = _case(T, hq, hkv, d, BF, 10)
    pos = torch.randint(0, 1 << 17, (1, T), device="cuda", dtype=torch.int32)
    _check(q, k, dy, dyk, gains, pos, rope.Rope(d, interleaved=inter))


def test_gains_of_any_place_and_type_in_autograd():
    q, k, dy, dyk, gains = _case(33, 2, 1, 64, BF, 11, "heads")
    pos, rp = torch.arange(33, device="cuda"), rope.Rope(64)
    store = torch.cat([torch.zeros(1, device="cuda"), *gains]).requires_grad_(True)
    a, b = rope.qk_norm_rope(q, k, pos, rp, store[1:65], store[65:])  # not 16-byte aligned
    (a.float() * dy.float()).sum().add((b.float() * dyk.float()).sum()).backward()
    *_, dgq, dgk = rope.qk_norm_rope_bwd(q, k, dy, dyk, pos, rp, *gains)
    assert torch.equal(store.grad[1:], torch.cat([dgq, dgk]))
    with pytest.raises(RuntimeError, match="ALIGNMENT"):
        rope.qk_norm_rope_fwd(q, k, pos, rp, store.detach()[1:65], gains[1])
