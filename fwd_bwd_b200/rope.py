"""QK-norm with rotary positions (include/sage_packed.h): argument marshalling only.

``qk_norm_rope`` normalizes every query and key vector over the head dimension, multiplies it by
a gain and rotates it by its token's position, in one pass over q and k, with autograd.  Its
outputs feed ``packed.packed_attention`` ([T, H, d] tensors) or ``ops.sage_attention`` with
``qknorm=False`` ([B, H, N, d] tensors).
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence, Tuple

import torch

from ._lib import SageRopeParams, SageRows, check, lib
from .ops import _DTYPES, _stream


class Rope:
    """The rotation and norm of one kind of layer: frequencies, axes and epsilon.

    Pair ``i`` of the first ``rotary_dim`` channels (all by default; a multiple of 16) is
    channels ``(i, i + rotary_dim/2)``, or ``(2i, 2i + 1)`` when ``interleaved``; its angle is
    ``position * inv_freq[i]``, by default ``inv_freq[i] = base^(-2i/rotary_dim)``.  With
    ``sections`` (pairs per axis, adding up to ``rotary_dim/2``, at most 4 axes) the first
    section's pairs turn by the first axis's positions, and so on (time, height, width of images
    and video).  ``norm=False`` rotates only; ``eps`` is the RMSNorm epsilon.
    """

    def __init__(self, d: int, base: float = 10000.0, rotary_dim: Optional[int] = None,
                 sections: Optional[Sequence[int]] = None, interleaved: bool = False,
                 inv_freq: Optional[Sequence[float]] = None, norm: bool = True,
                 eps: float = 1e-6):
        self.d = int(d)
        self.rotary_dim = self.d if rotary_dim is None else int(rotary_dim)
        if self.d not in (64, 128):
            raise ValueError("head dimension must be 64 or 128")
        if not 0 <= self.rotary_dim <= self.d or self.rotary_dim % 16:
            raise ValueError("rotary_dim must be a multiple of 16 between 0 and d")
        half = self.rotary_dim // 2
        if inv_freq is None:
            if not (math.isfinite(base) and base > 0):
                raise ValueError("base must be positive")
            inv_freq = [float(base) ** (-i / half) for i in range(half)]
        self.inv_freq = [float(f) for f in inv_freq]
        if len(self.inv_freq) != half or not all(math.isfinite(f) for f in self.inv_freq):
            raise ValueError(f"inv_freq must be {half} finite numbers")
        self.sections = [half] if sections is None else [int(s) for s in sections]
        if half and (len(self.sections) > 4 or min(self.sections, default=0) <= 0
                     or sum(self.sections) != half):
            raise ValueError(f"sections must be 1 to 4 positive numbers that add up to {half}")
        self.interleaved, self.norm, self.eps = bool(interleaved), bool(norm), float(eps)
        if not (math.isfinite(self.eps) and self.eps >= 0):
            raise ValueError("eps must be finite and not negative")
        self._freq = (ctypes.c_double * max(half, 1))(*self.inv_freq)
        self._sections = (ctypes.c_int * 4)(*(self.sections if half else []))

    @property
    def axes(self) -> int:
        return len(self.sections) if self.rotary_dim else 0


def _shape(x: torch.Tensor) -> Tuple[int, int, int, int]:
    """(B, N, H, d) of packed [T, H, d] or batched [B, H, N, d] vectors."""
    if x.dim() == 3:
        return (1, x.shape[0], x.shape[1], x.shape[2])
    if x.dim() == 4:
        return (x.shape[0], x.shape[2], x.shape[1], x.shape[3])
    raise ValueError("q and k must be [T, H, d] or [B, H, N, d]")


def _strides(x: torch.Tensor) -> Tuple[int, int, int]:
    """Batch, token and head strides (elements)."""
    s = x.stride()
    return (0, s[0], s[1]) if x.dim() == 3 else (s[0], s[2], s[1])


def _supported(x: torch.Tensor) -> bool:
    """Whether the kernels can read x as it is: contiguous 16-byte aligned channels, every other
    stride a multiple of 8 elements and at least d."""
    if x.stride(-1) != 1 or x.data_ptr() % 16:
        return False
    d = x.shape[-1]
    return all(n == 1 or (s >= d and s % 8 == 0)
               for n, s in zip(x.shape[:-1], x.stride()[:-1]))


def _rows(x: torch.Tensor) -> SageRows:
    return SageRows(x.data_ptr(), *_strides(x))


def _check_rows(name: str, x: torch.Tensor, like: Optional[torch.Tensor] = None) -> None:
    if not x.is_cuda:
        raise ValueError("libsage works on CUDA tensors only")
    if x.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float16 or bfloat16")
    if like is not None and (x.shape != like.shape or x.dtype != like.dtype
                             or x.device != like.device):
        raise ValueError(f"{name} must have the shape, type and device of the tensor it belongs to")
    if not _supported(x):
        raise ValueError(f"{name}: channels must be contiguous and 16-byte aligned, the other "
                         "strides multiples of 8 elements and at least d")


def _params(q, k, positions, rope: Rope, gains) -> Tuple[SageRopeParams, Optional[int]]:
    _check_rows("q", q)
    _check_rows("k", k)
    B, N, Hq, d = _shape(q)
    if q.dim() != k.dim() or q.dtype != k.dtype or q.device != k.device:
        raise ValueError("q and k must have one layout, type and device")
    Bk, Nk, Hkv, dk = _shape(k)
    if (Bk, Nk, dk) != (B, N, d) or d != rope.d:
        raise ValueError("q and k must hold the same tokens, with rope.d channels")
    for g in gains:
        if g is None:
            continue
        if not rope.norm:
            raise ValueError("gains belong to the norm (norm=False takes none)")
        if (g.dtype != torch.float32 or g.shape != (d,) or g.device != q.device
                or not g.is_contiguous()):
            raise ValueError("gains must be contiguous float32 [d] tensors on q's device")
    axis_stride = batch_stride = 0
    bits, ptr = 32, None
    if rope.rotary_dim:
        if positions is None:
            raise ValueError("positions are needed")
        if positions.dtype not in (torch.int32, torch.int64) or positions.device != q.device:
            raise ValueError("positions must be int32 or int64 on q's device")
        lead = () if rope.axes == 1 else (rope.axes,)
        shapes = [lead + (N,)] + ([lead + (B, N)] if q.dim() == 4 else [])
        if rope.axes == 1:
            shapes += [(1,) + s for s in shapes]
        if tuple(positions.shape) not in shapes or not positions.is_contiguous():
            raise ValueError(f"positions must be contiguous, of shape {shapes[0]}"
                             + (f" or {shapes[1]}" if q.dim() == 4 else ""))
        per_axis = positions.numel() // rope.axes
        axis_stride = per_axis
        batch_stride = N if per_axis == B * N and B > 1 else 0
        bits, ptr = (32 if positions.dtype == torch.int32 else 64), positions.data_ptr()
    prm = SageRopeParams(B, N, Hq, Hkv, d, _DTYPES[q.dtype], int(rope.norm), rope.eps,
                         rope.rotary_dim, int(rope.interleaved), rope.axes, rope._sections,
                         ctypes.cast(rope._freq, ctypes.c_void_p), bits, axis_stride,
                         batch_stride)
    return prm, ptr


def _ptr(x: Optional[torch.Tensor]) -> Optional[int]:
    return None if x is None else x.data_ptr()


def _out(name: str, x: Optional[torch.Tensor], like: torch.Tensor) -> torch.Tensor:
    if x is None:
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    _check_rows(name, x, like)
    return x


def qk_norm_rope_fwd(q, k, positions, rope: Rope, gain_q=None, gain_k=None, q_out=None,
                     k_out=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Normalized and rotated (q, k) (sage_qk_norm_rope_fwd).

    q, k: CUDA fp16/bf16 [T, H, d] or [B, H, N, d], any strides the kernels can read (slices of
    one projection); positions: int32/int64 [N] or, with several axes, [axes, N] (for batched q
    and k also [B, N] or [axes, B, N]); gains: float32 [d] or None for ones.  Outputs given by
    the caller must not overlap the inputs.
    """
    prm, pos = _params(q, k, positions, rope, (gain_q, gain_k))
    q_out, k_out = _out("q_out", q_out, q), _out("k_out", k_out, k)
    if prm.B * prm.N == 0:
        return q_out, k_out
    with torch.cuda.device(q.device):
        check("sage_qk_norm_rope_fwd", lib().sage_qk_norm_rope_fwd(
            ctypes.byref(prm), _rows(q), _rows(k), _ptr(gain_q), _ptr(gain_k), pos,
            _rows(q_out), _rows(k_out), _stream(q.device)))
    return q_out, k_out


def qk_norm_rope_bwd(q, k, dq_out, dk_out, positions, rope: Rope, gain_q=None, gain_k=None,
                     dq=None, dk=None, workspace: Optional[torch.Tensor] = None):
    """Gradients (dq, dk, dgain_q, dgain_k) given those of the outputs (sage_qk_norm_rope_bwd).

    The gains' gradients are float32 [d] whether or not gains were given (None without norm).
    """
    prm, pos = _params(q, k, positions, rope, (gain_q, gain_k))
    _check_rows("dq_out", dq_out, q)
    _check_rows("dk_out", dk_out, k)
    dq, dk = _out("dq", dq, q), _out("dk", dk, k)
    dgain = torch.empty((2, rope.d), dtype=torch.float32, device=q.device) if rope.norm else None
    if prm.B * prm.N == 0:
        if dgain is None:
            return dq, dk, None, None
        dgain.zero_()
        return dq, dk, dgain[0], dgain[1]
    if workspace is None and rope.norm:
        n = int(lib().sage_qk_norm_rope_workspace_bytes(ctypes.byref(prm)))
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    with torch.cuda.device(q.device):
        check("sage_qk_norm_rope_bwd", lib().sage_qk_norm_rope_bwd(
            ctypes.byref(prm), _rows(q), _rows(k), _ptr(gain_q), _ptr(gain_k), pos,
            _rows(dq_out), _rows(dk_out), _rows(dq), _rows(dk),
            dgain[0].data_ptr() if rope.norm else None,
            dgain[1].data_ptr() if rope.norm else None, _ptr(workspace),
            0 if workspace is None else workspace.numel() * workspace.element_size(),
            _stream(q.device)))
    return (dq, dk, dgain[0], dgain[1]) if rope.norm else (dq, dk, None, None)


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, rope, gain_q, gain_k):
        q = q if _supported(q) else q.contiguous()
        k = k if _supported(k) else k.contiguous()
        gains = [None if g is None else g.detach().float().contiguous() for g in (gain_q, gain_k)]
        ctx.save_for_backward(q, k, positions, *gains)
        ctx.rope = rope
        ctx.gain_dtypes = [None if g is None else g.dtype for g in (gain_q, gain_k)]
        return qk_norm_rope_fwd(q, k, positions, rope, *gains)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, positions, gq, gk = ctx.saved_tensors
        dq_out = dq_out if _supported(dq_out) else dq_out.contiguous()
        dk_out = dk_out if _supported(dk_out) else dk_out.contiguous()
        dq, dk, dgq, dgk = qk_norm_rope_bwd(q, k, dq_out, dk_out, positions, ctx.rope, gq, gk)
        dgains = [None if t is None else g.to(t) for g, t in zip((dgq, dgk), ctx.gain_dtypes)]
        return dq, dk, None, None, dgains[0], dgains[1]


def qk_norm_rope(q, k, positions, rope: Rope, gain_q=None, gain_k=None):
    """``qk_norm_rope_fwd`` with autograd, for q, k and the gains (of any floating type)."""
    return _QkNormRope.apply(q, k, positions, rope, gain_q, gain_k)


__all__ = ["Rope", "qk_norm_rope", "qk_norm_rope_bwd", "qk_norm_rope_fwd"]
