"""Calls of the packed operators that their documentation allows and that are easy to get wrong:
tensors off their alignment, tensors without heads."""
import pytest
import torch

from fwd_bwd_b200 import ops, packed, rope

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _off(x, by):
    """x's values in a contiguous view ``by`` elements behind a 16-byte boundary."""
    store = torch.zeros(x.numel() + by, dtype=x.dtype, device=x.device)
    y = store[by:].view(x.shape)
    y.copy_(x)
    assert y.is_contiguous() and y.data_ptr() % 16 == by * x.element_size()
    return y


def _random(T, h, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, h, d), generator=g, device="cuda").to(BF)


@pytest.mark.parametrize("by", [1, 4])
def test_attention_autograd_of_tensors_off_their_alignment(by):
    lengths = [150, 61]
    T = sum(lengths)
    x = [_random(T, h, 64, i) for i, h in enumerate((4, 2, 2, 4))]
    batch = packed.Batch(lengths)

    def run(q, k, v, do):
        leaves = [t.detach().requires_grad_(True) for t in (q, k, v)]
        o = packed.packed_attention(*leaves, batch)
        o.backward(do)
        return (o, *(t.grad for t in leaves))

    want = run(*x)
    for which in ([0], [1], [2], [3], [0, 1, 2, 3]):
        got = run(*(_off(t, by) if i in which else t for i, t in enumerate(x)))
        for a, b in zip(got, want):
            assert torch.equal(a, b), which
    assert ops.device_status() == 0


@pytest.mark.parametrize("by", [1, 4])
def test_rotary_autograd_of_tensors_off_their_alignment(by):
    T = 77
    x = [_random(T, h, 64, i) for i, h in enumerate((3, 2, 3, 2))]
    gains = [torch.rand(64, device="cuda") for _ in range(2)]
    pos, rp = torch.arange(T, device="cuda"), rope.Rope(64)

    def run(q, k, dq, dk):
        leaves = [t.detach().requires_grad_(True) for t in (q, k, *gains)]
        y = rope.qk_norm_rope(leaves[0], leaves[1], pos, rp, leaves[2], leaves[3])
        torch.autograd.backward(y, (dq, dk))
        return (*y, *(t.grad for t in leaves))

    want = run(*x)
    for which in ([0], [1], [2], [3], [0, 1, 2, 3]):
        got = run(*(_off(t, by) if i in which else t for i, t in enumerate(x)))
        for a, b in zip(got, want):
            assert torch.equal(a, b), which


def test_one_tensor_without_heads_is_refused():
    """Not taken for nothing to do, which would leave the other's outputs unwritten."""
    T, rp = 10, rope.Rope(64)
    some, none = _random(T, 2, 64, 0), _random(T, 0, 64, 0)
    pos = torch.arange(T, device="cuda")
    for q, k in ((none, some), (some, none)):
        with pytest.raises(ValueError, match="heads"):
            rope.qk_norm_rope_fwd(q, k, pos, rp)
        with pytest.raises(ValueError, match="heads"):
            rope.qk_norm_rope_bwd(q, k, q, k, pos, rp)
        with pytest.raises(ValueError, match="heads"):
            rope.qk_norm_rope(q[None].transpose(1, 2), k[None].transpose(1, 2), pos, rp)
    for x in rope.qk_norm_rope_fwd(none, none, pos, rp):
        assert x.shape == (T, 0, 64)
