"""Attention over packed sequences with grouped heads (include/sage_packed.h): argument
marshalling only.

Sequences of different lengths lie end to end in the rows of [T, H, d] tensors; a ``Batch`` holds
their lengths and the plan the kernels work from.  ``packed_attention`` is the autograd form,
``attn_fwd`` / ``attn_bwd`` the calls it makes.
"""
from __future__ import annotations

import ctypes
import operator
from typing import Optional, Sequence, Tuple

import torch

from ._lib import SageError, SagePackedInfo, SagePackedParams, check, lib
from ._lib import SAGE_ERR_INVALID_ARG
from .rope import _call, _like, _readable, _rows, _type_and_device


class Batch:
    """Sequences of ``lengths`` tokens (0 is allowed) laid end to end, on one device.

    ``lengths``: a sequence of ints or a CPU integer tensor.  The plan (a list of the sequences'
    tiles, largest work first) is made on the host and copied to the device once; keep the
    Batch for every layer and step on the same lengths.  Calls only read it.  Make it outside of
    graph captures (it waits for the copy) and keep it as long as a captured graph that uses it.
    """

    def __init__(self, lengths: Sequence[int], device="cuda"):
        if isinstance(lengths, torch.Tensor):
            if lengths.is_cuda:
                raise ValueError("lengths must be on the host")
            if lengths.is_floating_point() or lengths.dim() != 1:
                raise ValueError("lengths must be a 1-D sequence of integers")
            lengths = lengths.tolist()
        try:
            self.lengths = [operator.index(n) for n in lengths]
        except TypeError:
            raise ValueError("lengths must be a 1-D sequence of integers") from None
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
        self.plan_ptr = self.plan.data_ptr()
        self._stream = 0
        if self.plan.is_cuda:
            # complete before any stream reads it
            stream = torch.cuda.current_stream(self.plan.device)
            stream.synchronize()
            self._stream = stream.cuda_stream
        self.tokens = int(self.info.tokens)

    def __reduce__(self):
        """Copies are made anew: a plan of their own, complete before they are used."""
        return type(self), (self.lengths, self.device)

    def _used_on(self, stream: torch.cuda.Stream) -> None:
        """Keeps the plan's memory from its allocating stream while another one reads it."""
        if stream.cuda_stream != self._stream:
            self.plan.record_stream(stream)

    @property
    def device(self) -> torch.device:
        return self.plan.device

    def positions(self) -> torch.Tensor:
        """int32 [tokens] on the batch's device: each token's index within its sequence."""
        return torch.cat([torch.arange(n, dtype=torch.int32) for n in self.lengths]).to(self.device)


def _params(q, k, v, batch: Batch, causal: bool, softmax_scale: float) -> SagePackedParams:
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v must be [T, H, d]")
    dtype, dev = _type_and_device(q)
    (T, Hq, d), (Tk, Hkv, dk) = q.shape, k.shape
    if k.shape != v.shape or Tk != T or dk != d:
        raise ValueError("q, k and v must hold the same tokens and channels, k and v the same "
                         "heads")
    if (q.dtype != k.dtype or q.dtype != v.dtype or k.get_device() != dev
            or v.get_device() != dev):
        raise ValueError("q, k and v must have one type and device")
    if Hkv == 0 or Hq % Hkv:
        raise ValueError("the query heads must be a multiple of the key heads")
    if T < batch.tokens:
        raise ValueError(f"the batch holds {batch.tokens} tokens, the tensors {T} rows")
    return SagePackedParams(T, Hq, Hkv, d, dtype, bool(causal), softmax_scale)


def _new(like: torch.Tensor, batch: Batch) -> torch.Tensor:
    """An output for ``like``'s shape whose rows behind the last sequence are zero."""
    x = torch.empty_like(like, memory_format=torch.contiguous_format)
    if like.shape[0] > batch.tokens:
        x[batch.tokens:].zero_()
    return x


def _check_lse(lse: torch.Tensor, q: torch.Tensor) -> None:
    if (lse.dtype != torch.float32 or lse.shape != (q.shape[1], q.shape[0])
            or lse.get_device() != q.get_device() or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [Hq, T] tensor on q's device")


def _check_batch(q: torch.Tensor, batch: Batch) -> None:
    if batch.plan.get_device() != q.get_device():
        raise ValueError("the batch must be on q's device")


def attn_fwd(q, k, v, batch: Batch, causal: bool = True, softmax_scale: float = 0.0, o=None,
             lse=None, workspace: Optional[torch.Tensor] = None
             ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention within each sequence (sage_packed_attn_fwd): (o [T, Hq, d], lse [Hq, T]).

    q: [T, Hq, d], k and v: [T, Hkv, d], CUDA fp16/bf16, 16-byte aligned, with any strides the
    kernels can read (slices of one projection); query head h reads key head h // (Hq / Hkv).  ``softmax_scale <= 0``
    selects 1/sqrt(d).  Sequences never touch each other, not even through NaN.  A row that sees a
    score of NaN or +inf is NaN in ``o`` and ``lse``; one of -inf weighs nothing.  A
    hidden key weighs exactly zero, so NaN or infinity in its v reaches the rows of its tile of 128
    tokens (cut from the sequence's end) as 0 * inf; rows of earlier tiles do not see it.
    Rows behind the last sequence of ``o`` and ``lse`` are left as they are
    when the caller gives them, zero otherwise.  Given outputs must not overlap the inputs.
    ``workspace``: a uint8 tensor of at least ``fwd_workspace_bytes`` elements (often none); calls
    that share one must be ordered.
    """
    prm = _params(q, k, v, batch, causal, softmax_scale)
    _check_batch(q, batch)
    o = _new(q, batch) if o is None else o
    if lse is None:
        lse = q.new_empty((prm.Hq, prm.T), dtype=torch.float32)
        if prm.T > batch.tokens:
            lse[:, batch.tokens:].zero_()
    else:
        _check_lse(lse, q)
    rows_o = _like("o", o, q)
    if batch.tokens:
        if workspace is None:
            n = int(lib().sage_packed_attn_fwd_workspace_bytes(prm, batch.info))
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
        else:
            _check_workspace(workspace, q)
        _call("sage_packed_attn_fwd", q.get_device(), batch._used_on, prm, batch.info,
              batch.plan_ptr, _rows(q), _rows(k), _rows(v), rows_o, lse.data_ptr(),
              *_workspace_args(workspace))
    return o, lse


def attn_bwd(q, k, v, o, lse, dout, batch: Batch, causal: bool = True, softmax_scale: float = 0.0,
             dq=None, dk=None, dv=None, workspace: Optional[torch.Tensor] = None):
    """Gradients (dq, dk, dv) from the forward's o and lse and o's gradient (sage_packed_attn_bwd).

    Rows behind the last sequence as in ``attn_fwd``.  ``workspace``: a uint8 tensor of at least
    ``workspace_bytes`` elements; calls that share one must be ordered.
    """
    prm = _params(q, k, v, batch, causal, softmax_scale)
    rows = (_rows(q), _rows(k), _rows(v), _like("o", o, q))
    rows_do = _like("dout", dout, q)
    _check_batch(q, batch)
    _check_lse(lse, q)
    dq = _new(q, batch) if dq is None else dq
    dk = _new(k, batch) if dk is None else dk
    dv = _new(v, batch) if dv is None else dv
    grads = (_like("dq", dq, q), _like("dk", dk, k), _like("dv", dv, k))
    if batch.tokens == 0:
        return dq, dk, dv
    if workspace is None:
        workspace = torch.empty(_workspace_bytes(prm, batch), dtype=torch.uint8, device=q.device)
    else:
        _check_workspace(workspace, q)
    _call("sage_packed_attn_bwd", q.get_device(), batch._used_on, prm, batch.info, batch.plan_ptr,
          *rows, lse.data_ptr(), rows_do, *grads, *_workspace_args(workspace))
    return dq, dk, dv


def _check_workspace(workspace: torch.Tensor, q: torch.Tensor) -> None:
    if workspace.get_device() != q.get_device() or not workspace.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on q's device")


def _workspace_args(workspace: Optional[torch.Tensor]) -> Tuple[Optional[int], int]:
    if workspace is None:
        return None, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _workspace_bytes(prm: SagePackedParams, batch: Batch) -> int:
    return int(lib().sage_packed_attn_bwd_workspace_bytes(prm, batch.info))


def workspace_bytes(q, k, v, batch: Batch, causal: bool = True) -> int:
    """Bytes of scratch ``attn_bwd`` needs on these tensors."""
    return _workspace_bytes(_params(q, k, v, batch, causal, 0.0), batch)


def fwd_workspace_bytes(q, k, v, batch: Batch, causal: bool = True) -> int:
    """Bytes of scratch ``attn_fwd`` needs on these tensors (0 for most)."""
    prm = _params(q, k, v, batch, causal, 0.0)
    return int(lib().sage_packed_attn_fwd_workspace_bytes(prm, batch.info))


class _PackedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, batch, causal, softmax_scale):
        q, k, v = (_readable(x) for x in (q, k, v))
        o, lse = attn_fwd(q, k, v, batch, causal, softmax_scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.args = (batch, causal, softmax_scale)
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        q, k, v, o, lse = ctx.saved_tensors
        dq, dk, dv = attn_bwd(q, k, v, o, lse, _readable(dout), *ctx.args)
        return dq, dk, dv, None, None, None


def packed_attention(q, k, v, batch: Batch, causal: bool = True, softmax_scale: float = 0.0):
    """``attn_fwd`` with autograd: o [T, Hq, d].  Tensors and gradients that the kernels cannot read
    where they are (off a 16-byte boundary, or with other strides) are copied."""
    return _PackedAttention.apply(q, k, v, batch, causal, softmax_scale)


__all__ = ["Batch", "attn_bwd", "attn_fwd", "fwd_workspace_bytes", "packed_attention",
           "workspace_bytes"]
