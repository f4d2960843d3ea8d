"""Attention over packed sequences with grouped heads (include/sage_packed.h): argument
marshalling only.

Sequences of different lengths lie end to end in the rows of [T, H, d] tensors; a ``Batch`` holds
their lengths and the plan the kernels work from.  ``packed_attention`` is the autograd form,
``attn_fwd`` / ``attn_bwd`` the calls it makes.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple

import torch

from ._lib import SageError, SagePackedInfo, SagePackedParams, check, lib
from ._lib import SAGE_ERR_INVALID_ARG
from .ops import _DTYPES, _stream
from .rope import _check_rows, _rows, _supported


class Batch:
    """Sequences of ``lengths`` tokens (0 is allowed) laid end to end, on one device.

    ``lengths``: a sequence of ints or a CPU integer tensor.  The plan (a list of the sequences'
    tiles, largest work first) is made on the host and copied to the device once; keep the
    Batch for every layer and step on the same lengths.  Calls only read it.
    """

    def __init__(self, lengths: Sequence[int], device="cuda"):
        if isinstance(lengths, torch.Tensor):
            if lengths.is_cuda:
                raise ValueError("lengths must be on the host")
            if lengths.is_floating_point() or lengths.dim() != 1:
                raise ValueError("lengths must be a 1-D sequence of integers")
            lengths = lengths.tolist()
        self.lengths = [int(n) for n in lengths]
        if not self.lengths or min(self.lengths) < 0 or max(self.lengths) >= 2 ** 31:
            raise ValueError("lengths must be a non-empty sequence of integers >= 0")
        arr = (ctypes.c_int * len(self.lengths))(*self.lengths)
        n = int(lib().sage_packed_plan_bytes(arr, len(self.lengths)))
        if n == 0:
            raise SageError("sage_packed_plan_bytes", SAGE_ERR_INVALID_ARG,
                            "the sequences hold too many tokens")
        host = torch.empty(n, dtype=torch.uint8)
        self.info = SagePackedInfo()
        check("sage_packed_plan_fill", lib().sage_packed_plan_fill(
            arr, len(self.lengths), host.data_ptr(), n, ctypes.byref(self.info)))
        self.plan = host.to(torch.device(device))
        self.tokens = int(self.info.tokens)

    @property
    def device(self) -> torch.device:
        return self.plan.device

    def positions(self) -> torch.Tensor:
        """int32 [tokens] on the batch's device: each token's index within its sequence."""
        return torch.cat([torch.arange(n, dtype=torch.int32) for n in self.lengths]).to(self.device)


def _params(q, k, v, batch: Batch, causal: bool, softmax_scale: float) -> SagePackedParams:
    for name, x in (("q", q), ("k", k), ("v", v)):
        if x.dim() != 3:
            raise ValueError(f"{name} must be [T, H, d]")
        _check_rows(name, x)
    if k.shape != v.shape or k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
        raise ValueError("q, k and v must hold the same tokens and channels, k and v the same heads")
    if not (q.dtype == k.dtype == v.dtype and q.device == k.device == v.device == batch.device):
        raise ValueError("q, k, v and the batch must have one type and device")
    T, Hq, d = q.shape
    if k.shape[1] == 0 or Hq % k.shape[1]:
        raise ValueError("the query heads must be a multiple of the key heads")
    if T < batch.tokens:
        raise ValueError(f"the batch holds {batch.tokens} tokens, the tensors {T} rows")
    return SagePackedParams(T, Hq, k.shape[1], d, _DTYPES[q.dtype], int(causal),
                            float(softmax_scale))


def _out(name: str, x: Optional[torch.Tensor], like: torch.Tensor, batch: Batch) -> torch.Tensor:
    """The caller's output, or a new one whose rows behind the last sequence are zero."""
    if x is None:
        x = torch.empty(like.shape, dtype=like.dtype, device=like.device)
        if like.shape[0] > batch.tokens:
            x[batch.tokens:].zero_()
        return x
    _check_rows(name, x, like)
    return x


def _check_lse(lse: torch.Tensor, q: torch.Tensor) -> None:
    if (lse.dtype != torch.float32 or lse.shape != (q.shape[1], q.shape[0])
            or lse.device != q.device or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [Hq, T] tensor on q's device")


def attn_fwd(q, k, v, batch: Batch, causal: bool = True, softmax_scale: float = 0.0, o=None,
             lse=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention within each sequence (sage_packed_attn_fwd): (o [T, Hq, d], lse [Hq, T]).

    q: [T, Hq, d], k and v: [T, Hkv, d], CUDA fp16/bf16, any strides the kernels can read (slices
    of one projection); query head h reads key head h // (Hq / Hkv).  ``softmax_scale <= 0``
    selects 1/sqrt(d).  Rows behind the last sequence of ``o`` and ``lse`` are left as they are
    when the caller gives them, zero otherwise.  Given outputs must not overlap the inputs.
    """
    prm = _params(q, k, v, batch, causal, softmax_scale)
    o = _out("o", o, q, batch)
    if lse is None:
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
        if q.shape[0] > batch.tokens:
            lse[:, batch.tokens:].zero_()
    _check_lse(lse, q)
    if batch.tokens == 0:
        return o, lse
    with torch.cuda.device(q.device):
        check("sage_packed_attn_fwd", lib().sage_packed_attn_fwd(
            ctypes.byref(prm), ctypes.byref(batch.info), batch.plan.data_ptr(), _rows(q),
            _rows(k), _rows(v), _rows(o), lse.data_ptr(), _stream(q.device)))
    return o, lse


def attn_bwd(q, k, v, o, lse, dout, batch: Batch, causal: bool = True, softmax_scale: float = 0.0,
             dq=None, dk=None, dv=None, workspace: Optional[torch.Tensor] = None):
    """Gradients (dq, dk, dv) from the forward's o and lse and o's gradient (sage_packed_attn_bwd).

    Rows behind the last sequence as in ``attn_fwd``.  ``workspace``: a uint8 tensor of at least
    ``workspace_bytes`` elements; calls that share one must be ordered.
    """
    prm = _params(q, k, v, batch, causal, softmax_scale)
    _check_rows("o", o, q)
    _check_rows("dout", dout, q)
    _check_lse(lse, q)
    dq, dk, dv = (_out(n, x, like, batch)
                  for n, x, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)))
    if batch.tokens == 0:
        return dq, dk, dv
    if workspace is None:
        workspace = torch.empty(_workspace_bytes(prm, batch), dtype=torch.uint8, device=q.device)
    elif workspace.device != q.device or not workspace.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on q's device")
    with torch.cuda.device(q.device):
        check("sage_packed_attn_bwd", lib().sage_packed_attn_bwd(
            ctypes.byref(prm), ctypes.byref(batch.info), batch.plan.data_ptr(), _rows(q),
            _rows(k), _rows(v), _rows(o), lse.data_ptr(), _rows(dout), _rows(dq), _rows(dk),
            _rows(dv), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            _stream(q.device)))
    return dq, dk, dv


def _workspace_bytes(prm: SagePackedParams, batch: Batch) -> int:
    return int(lib().sage_packed_attn_bwd_workspace_bytes(ctypes.byref(prm),
                                                          ctypes.byref(batch.info)))


def workspace_bytes(q, k, v, batch: Batch) -> int:
    """Bytes of scratch ``attn_bwd`` needs on these tensors."""
    return _workspace_bytes(_params(q, k, v, batch, True, 0.0), batch)


class _PackedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, batch, causal, softmax_scale):
        q, k, v = (x if _supported(x) else x.contiguous() for x in (q, k, v))
        o, lse = attn_fwd(q, k, v, batch, causal, softmax_scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.args = (batch, causal, softmax_scale)
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        q, k, v, o, lse = ctx.saved_tensors
        dout = dout if _supported(dout) else dout.contiguous()
        dq, dk, dv = attn_bwd(q, k, v, o, lse, dout, *ctx.args)
        return dq, dk, dv, None, None, None


def packed_attention(q, k, v, batch: Batch, causal: bool = True, softmax_scale: float = 0.0):
    """``attn_fwd`` with autograd: o [T, Hq, d]."""
    return _PackedAttention.apply(q, k, v, batch, causal, softmax_scale)


__all__ = ["Batch", "attn_bwd", "attn_fwd", "packed_attention", "workspace_bytes"]
