"""Host side of the packed operators' arguments (no GPU)."""
import copy
import ctypes
import pickle

import numpy as np
import pytest
import torch

from fwd_bwd_b200 import packed, rope


def test_copies_only_what_the_kernels_cannot_read():
    store = torch.randn(4 * 3 * 64 + 8).bfloat16()
    x = store[:4 * 3 * 64].view(4, 3, 64)
    assert x.data_ptr() % 16 == 0
    for same in (x, x[:, 1:], x[::2], x.transpose(0, 1), x[:1], x[:0]):
        assert rope._readable(same) is same
    off = store[1:1 + 4 * 3 * 64].view(4, 3, 64)
    for y in (off, off[:, 1:], off[:, 1:2], off.transpose(0, 1), x[..., :1].expand(-1, -1, 64),
              x[:, :1].expand(-1, 3, -1), x.transpose(1, 2).contiguous().transpose(1, 2)):
        z = rope._readable(y)
        assert torch.equal(z, y) and rope._supported(z)
        assert z.data_ptr() % 16 == 0 and z.data_ptr() != y.data_ptr()


@pytest.mark.parametrize("lengths", [[2.5], [3.0, 1], np.array([2.0, 7.9]), ["4"], [None]], ids=str)
def test_lengths_that_are_not_integers_are_refused(lengths):
    with pytest.raises(ValueError, match="integers"):
        packed.Batch(lengths, device="cpu")


def test_lengths_of_every_integer_type():
    for lengths in (np.array([3, 0, 5]), np.array([3, 0, 5], np.uint8), (3, 0, 5),
                    torch.tensor([3, 0, 5]), list(torch.tensor([3, 0, 5], dtype=torch.int32))):
        assert packed.Batch(lengths, device="cpu").lengths == [3, 0, 5]


def _copies(x):
    return copy.copy(x), copy.deepcopy(x), pickle.loads(pickle.dumps(x))


def test_copies_of_a_batch_use_their_own_plan():
    b = packed.Batch([300, 0, 5], device="cpu")
    for c in _copies(b):
        assert c.plan_ptr == c.plan.data_ptr()
        assert c.lengths == b.lengths and c.tokens == b.tokens and torch.equal(c.plan, b.plan)
        assert bytes(c.info) == bytes(b.info) and c.device == b.device
        assert c.positions().tolist() == b.positions().tolist()


def test_copies_of_a_rope_use_their_own_frequencies():
    r = rope.Rope(64, rotary_dim=32, sections=[5, 11], interleaved=True, eps=1e-5)
    for c in _copies(r):
        assert c._freq_ptr == ctypes.addressof(c._freq)
        assert list(c._freq) == r.inv_freq == c.inv_freq and list(c._sections) == [5, 11, 0, 0]
        assert (c.d, c.rotary_dim, c.axes, c.interleaved, c.norm, c.eps) == (64, 32, 2, True, True,
                                                                             1e-5)
