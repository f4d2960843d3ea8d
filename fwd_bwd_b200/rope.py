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
from .ops import _DTYPES


class Rope:
    """The rotation and norm of one kind of layer: frequencies, axes and epsilon.

    Pair ``i`` of the first ``rotary_dim`` channels (all by default; a multiple of 16) is
    channels ``(i, i + rotary_dim/2)``, or ``(2i, 2i + 1)`` when ``interleaved``; its angle is
    ``position * inv_freq[i]``, by default ``inv_freq[i] = base^(-2i/rotary_dim)``.  With
    ``sections`` (pairs per axis, adding up to ``rotary_dim/2``, at most 4 axes) the first
    section's pairs turn by the first axis's positions, and so on (time, height, width of images
    and video).  ``norm=False`` rotates only; ``eps`` is the RMSNorm epsilon.  Angles keep their
    accuracy (2^-20) up to positions of 2^40; beyond, they are off by up to 2 pi |position| 2^-64.
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
        self._freq_ptr = ctypes.addressof(self._freq)
        self._sections = (ctypes.c_int * 4)(*(self.sections if half else []))

    def __reduce__(self):
        """Copies are made anew: the library reads frequencies at an address of their own."""
        return type(self), (self.d, 1.0, self.rotary_dim, self.sections if self.rotary_dim else None,
                            self.interleaved, self.inv_freq, self.norm, self.eps)

    @property
    def axes(self) -> int:
        return len(self.sections) if self.rotary_dim else 0


def _supported(x: torch.Tensor) -> bool:
    """Whether the kernels can read x as it is: contiguous 16-byte aligned channels, every other
    stride a multiple of 8 elements and at least d."""
    if x.stride(-1) != 1 or x.data_ptr() % 16:
        return False
    d = x.shape[-1]
    return all(n == 1 or (s >= d and s % 8 == 0)
               for n, s in zip(x.shape[:-1], x.stride()[:-1]))


def _readable(x: torch.Tensor) -> torch.Tensor:
    """x, or a copy of it where the kernels cannot read it as it is."""
    if _supported(x):
        return x
    y = x.contiguous()  # x itself when only its address is off
    return y if _supported(y) else y.clone()


def _rows(x: torch.Tensor) -> SageRows:
    """The tensor's description for the C ABI, which checks pointers, alignment, the other strides
    and overlap within an output."""
    s = x.stride()
    if s[-1] != 1:
        raise ValueError("channels must be contiguous")
    if len(s) == 3:
        return SageRows(x.data_ptr(), 0, s[0], s[1])
    return SageRows(x.data_ptr(), s[0], s[2], s[1])


def _new(like: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(like, memory_format=torch.contiguous_format)


def _like(name: str, x: torch.Tensor, like: torch.Tensor) -> SageRows:
    """``_rows`` of a tensor that belongs to ``like``."""
    if x.shape != like.shape or x.dtype != like.dtype or x.get_device() != like.get_device():
        raise ValueError(f"{name} must have the shape, type and device of the tensor it belongs to")
    return _rows(x)


def _type_and_device(x: torch.Tensor) -> Tuple[int, int]:
    dev, dtype = x.get_device(), _DTYPES.get(x.dtype)
    if dev < 0:
        raise ValueError("libsage works on CUDA tensors only")
    if dtype is None:
        raise ValueError("tensors must be float16 or bfloat16")
    return dtype, dev


def _params(q, k, positions, rope: Rope, gains) -> Tuple[SageRopeParams, Optional[int]]:
    dtype, dev = _type_and_device(q)
    qs, ks = q.shape, k.shape
    if len(qs) == 3:
        B, (N, Hq, d), Hkv = 1, qs, ks[1]
    elif len(qs) == 4:
        B, Hq, N, d = qs
        Hkv = ks[1]
    else:
        raise ValueError("q and k must be [T, H, d] or [B, H, N, d]")
    if len(ks) != len(qs) or q.dtype != k.dtype or k.get_device() != dev:
        raise ValueError("q and k must have one layout, type and device")
    if (ks[0] != qs[0] or ks[-1] != d or d != rope.d or (len(qs) == 4 and ks[2] != N)):
        raise ValueError("q and k must hold the same tokens, with rope.d channels")
    if (Hq == 0) != (Hkv == 0) and B * N:
        raise ValueError("q and k must both have heads")
    for g in gains:
        if g is None:
            continue
        if not rope.norm:
            raise ValueError("gains belong to the norm (norm=False takes none)")
        if (g.dtype != torch.float32 or g.shape != (d,) or g.get_device() != dev
                or g.stride(0) != 1):
            raise ValueError("gains must be contiguous float32 [d] tensors on q's device")
    axis_stride = batch_stride = 0
    bits, ptr = 32, None
    if rope.rotary_dim:
        if positions is None:
            raise ValueError("positions are needed")
        bits = 32 if positions.dtype == torch.int32 else 64
        if (bits == 64 and positions.dtype != torch.int64) or positions.get_device() != dev:
            raise ValueError("positions must be int32 or int64 on q's device")
        ps, axes = tuple(positions.shape), rope.axes
        if axes == 1 and len(ps) > 1 and ps[0] == 1 and (len(qs) == 3 or ps != (B, N)):
            ps = ps[1:]  # [1, N] or [1, B, N]
        shared, own = ((N,), (B, N)) if axes == 1 else ((axes, N), (axes, B, N))
        if (ps != shared and (len(qs) != 4 or ps != own)) or not positions.is_contiguous():
            raise ValueError(f"positions must be contiguous, of shape {shared}"
                             + (f" or {own}" if len(qs) == 4 else ""))
        axis_stride = N if ps == shared else B * N
        batch_stride = 0 if ps == shared else N
        ptr = positions.data_ptr()
    prm = SageRopeParams(B, N, Hq, Hkv, d, dtype, rope.norm, rope.eps,
                         rope.rotary_dim, rope.interleaved, rope.axes, rope._sections,
                         rope._freq_ptr, bits, axis_stride, batch_stride)
    return prm, ptr


def _ptr(x: Optional[torch.Tensor]) -> Optional[int]:
    return None if x is None else x.data_ptr()


def _call(name: str, device: int, used_on, *args) -> None:
    """Calls the library on the tensors' device and its current stream, of which ``used_on`` (or
    None) is told."""
    stream = torch.cuda.current_stream(device)
    if used_on is not None:
        used_on(stream)
    stream = stream.cuda_stream
    if torch.cuda.current_device() == device:
        status = getattr(lib(), name)(*args, stream)
    else:
        with torch.cuda.device(device):
            status = getattr(lib(), name)(*args, stream)
    if status:
        check(name, status)


def qk_norm_rope_fwd(q, k, positions, rope: Rope, gain_q=None, gain_k=None, q_out=None,
                     k_out=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Normalized and rotated (q, k) (sage_qk_norm_rope_fwd).

    q, k: CUDA fp16/bf16 [T, H, d] or [B, H, N, d], any strides the kernels can read (slices of
    one projection); positions: int32/int64 [N] or, with several axes, [axes, N] (for batched q
    and k also [B, N] or [axes, B, N]); gains: float32 [d], 16-byte aligned, or None for ones.
    Outputs given by the caller must not overlap the inputs.
    """
    prm, pos = _params(q, k, positions, rope, (gain_q, gain_k))
    q_out = _new(q) if q_out is None else q_out
    k_out = _new(k) if k_out is None else k_out
    rows_q, rows_k = _like("q_out", q_out, q), _like("k_out", k_out, k)
    if q.numel():
        _call("sage_qk_norm_rope_fwd", q.get_device(), None, prm, _rows(q), _rows(k), _ptr(gain_q),
              _ptr(gain_k), pos, rows_q, rows_k)
    return q_out, k_out


def qk_norm_rope_bwd(q, k, dq_out, dk_out, positions, rope: Rope, gain_q=None, gain_k=None,
                     dq=None, dk=None, workspace: Optional[torch.Tensor] = None):
    """Gradients (dq, dk, dgain_q, dgain_k) given those of the outputs (sage_qk_norm_rope_bwd).

    The gains' gradients are float32 [d] whether or not gains were given (None without norm).
    """
    prm, pos = _params(q, k, positions, rope, (gain_q, gain_k))
    dq = _new(q) if dq is None else dq
    dk = _new(k) if dk is None else dk
    rows = (_like("dq_out", dq_out, q), _like("dk_out", dk_out, k), _like("dq", dq, q),
            _like("dk", dk, k))
    dgain_q = dgain_k = None
    if rope.norm:
        dgain_q, dgain_k = torch.empty((2, rope.d), dtype=torch.float32, device=q.device)
    if q.numel() == 0:
        if rope.norm:
            dgain_q.zero_()
            dgain_k.zero_()
        return dq, dk, dgain_q, dgain_k
    if workspace is None and rope.norm:
        n = int(lib().sage_qk_norm_rope_workspace_bytes(prm))
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    elif workspace is not None and (workspace.get_device() != q.get_device()
                                    or not workspace.is_contiguous()):
        raise ValueError("the workspace must be a contiguous tensor on q's device")
    _call("sage_qk_norm_rope_bwd", q.get_device(), None, prm, _rows(q), _rows(k), _ptr(gain_q),
          _ptr(gain_k), pos, *rows, _ptr(dgain_q), _ptr(dgain_k), _ptr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size())
    return dq, dk, dgain_q, dgain_k


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, rope, gain_q, gain_k):
        q, k = _readable(q), _readable(k)
        gains = [None if g is None else g.detach().float().contiguous() for g in (gain_q, gain_k)]
        gains = [g if g is None or g.data_ptr() % 16 == 0 else g.clone() for g in gains]
        ctx.save_for_backward(q, k, positions, *gains)
        ctx.rope = rope
        ctx.gain_dtypes = [None if g is None else g.dtype for g in (gain_q, gain_k)]
        return qk_norm_rope_fwd(q, k, positions, rope, *gains)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, positions, gq, gk = ctx.saved_tensors
        dq, dk, dgq, dgk = qk_norm_rope_bwd(q, k, _readable(dq_out), _readable(dk_out), positions,
                                            ctx.rope, gq, gk)
        dgains = [None if t is None else g.to(t) for g, t in zip((dgq, dgk), ctx.gain_dtypes)]
        return dq, dk, None, None, dgains[0], dgains[1]


def qk_norm_rope(q, k, positions, rope: Rope, gain_q=None, gain_k=None):
    """``qk_norm_rope_fwd`` with autograd, for q, k and the gains (of any floating type).  Tensors and
    gradients that the kernels cannot read where they are (off a 16-byte boundary, or with other
    strides) are copied."""
    return _QkNormRope.apply(q, k, positions, rope, gain_q, gain_k)


__all__ = ["Rope", "qk_norm_rope", "qk_norm_rope_bwd", "qk_norm_rope_fwd"]
