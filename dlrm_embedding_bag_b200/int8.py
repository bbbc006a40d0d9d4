"""Python binding of the 8-bit layers (the C ABI in ``include/dlrm_int8.h``).

Argument marshalling only, as in :mod:`.tokens`. A matrix in 8 bits is a pair
``(q, scale)``: int8 ``(rows, cols)`` with unit column stride and a row pitch
that is a multiple of 16 (:func:`int8_empty` makes such buffers), and one f32
scale for each row; its values are ``q * scale[:, None]``.

:func:`quantize_rows` rounds activations or weights, :func:`rms_norm_int8` does
it behind a root-mean-square norm of ``x + residual``, and :func:`linear_int8`
is the layer that multiplies the two. ``mlp.MLP(mode="int8")`` chains them.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import ops
from .mlp import ACTS
from .tokens import _call, _empty, _empty_vector, _flat, _lib, _matrix, _on, _pitch, _status

MAX_K = 131071

_norm = _lib.dlrm_rms_norm_int8
_quantize = _lib.dlrm_quantize_int8
_dequantize = _lib.dlrm_dequantize_int8
_linear = _lib.dlrm_linear_int8


def int8_empty(rows: int, cols: int, device="cuda") -> torch.Tensor:
    """A ``(rows, cols)`` int8 view whose row pitch is ``cols`` rounded up to 16."""
    t = torch.empty((rows, (cols + 15) // 16 * 16), dtype=torch.int8, device=device)
    return t if cols % 16 == 0 else t[:, :cols]


def _int8(t: torch.Tensor, name: str, index: Optional[int]) -> Tuple[int, int, int]:
    """(rows, columns, row pitch) of an int8 matrix."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is torch.int8) or \
            (index is not None and t.get_device() != index):
        _on(t, name, index)
        raise TypeError(f"{name} must be torch.int8 (got {t.dtype})")
    return _pitch(t, name)


def _scales(t: torch.Tensor, name: str, n: int, index: int) -> int:
    p = _flat(t, name, torch.float32, index)
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements (got {t.numel()})")
    return p


def _outputs(x, M, K, out, scale_out, index):
    """(out, scale_out, out's pitch): the 8-bit matrix and its scales, made where not given."""
    if out is None:
        pitch = (K + 15) // 16 * 16
        out = _empty(M, pitch, torch.int8, index)
        if pitch != K:
            out = out[:, :K]
    else:
        rows, cols, pitch = _int8(out, "out", index)
        if rows != M or cols != K:
            raise ValueError(f"out must be ({M}, {K}) (got {tuple(out.shape)})")
    if scale_out is None:
        scale_out = _empty_vector(M, torch.float32, index)
    else:
        _scales(scale_out, "scale_out", M, index)
    return out, scale_out, pitch


def quantize_rows(x: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                  scale_out: Optional[torch.Tensor] = None):
    """``(q, scale)`` of an f32 or bf16 ``(M, K)`` matrix: ``scale = max|row| / 127`` and
    ``q = row / scale`` rounded to nearest even. For weights ``(N, K)`` this is
    one scale for each output channel."""
    index, xd, M, K, ldx = _matrix(x, "x")
    out, scale_out, ldq = _outputs(x, M, K, out, scale_out, index)
    _call(_quantize, "dlrm_quantize_int8", index,
          (x.data_ptr(), ldx, xd, M, K, out.data_ptr(), ldq, scale_out.data_ptr()))
    return out, scale_out


def rms_norm_int8(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *,
                  residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  out: Optional[torch.Tensor] = None, scale_out: Optional[torch.Tensor] = None,
                  residual_out: Optional[torch.Tensor] = None):
    """Root-mean-square norm of ``h = x + residual`` in 8 bits; returns ``(q, scale, h)``.

    ``x`` and ``residual`` are f32 or bf16 ``(M, K)`` of one type, ``weight`` f32
    ``(K,)`` or None for ones. ``q * scale`` stands for
    ``h * weight / sqrt(mean(h^2) + eps)``; ``h`` is rounded once to the type of
    ``x`` into ``residual_out`` (which may be ``residual`` itself) or a new tensor,
    and is None without a residual.
    """
    index, xd, M, K, ldx = _matrix(x, "x")
    pr, ldr, ph, ldh = None, 0, None, 0
    if residual is not None:
        _on(residual, "residual", index)
        if residual.dtype != x.dtype or residual.shape != x.shape:
            raise ValueError(f"residual must be {x.dtype} ({M}, {K})")
        pr, ldr = residual.data_ptr(), _pitch(residual, "residual")[2]
        if residual_out is None:
            residual_out = _empty(M, K, x.dtype, index)
            ldh = K
        else:
            _on(residual_out, "residual_out", index)
            if residual_out.dtype != x.dtype or residual_out.shape != x.shape:
                raise ValueError(f"residual_out must be {x.dtype} ({M}, {K})")
            ldh = _pitch(residual_out, "residual_out")[2]
        ph = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs residual")
    pw = _scales(weight, "weight", K, index) if weight is not None else None
    out, scale_out, ldq = _outputs(x, M, K, out, scale_out, index)
    _call(_norm, "dlrm_rms_norm_int8", index,
          (x.data_ptr(), ldx, pr, ldr, xd, pw, M, K, eps, ph, ldh, out.data_ptr(), ldq,
           scale_out.data_ptr()))
    return out, scale_out, residual_out


def dequantize_rows(q: torch.Tensor, scale: torch.Tensor, *,
                    dtype: torch.dtype = torch.float32,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of a matrix in 8 bits, ``q * scale[:, None]``, rounded once to ``dtype``."""
    M, K, ldq = _int8(q, "q", None)
    index = q.get_device()
    ps = _scales(scale, "scale", M, index)
    if out is None:
        od, ldo = ops.TABLE_DTYPES.get(dtype), K
        if od is None:
            raise TypeError(f"dtype must be float32 or bfloat16 (got {dtype})")
        out = _empty(M, K, dtype, index)
    else:
        _, od, rows, cols, ldo = _matrix(out, "out", index)
        if rows != M or cols != K:
            raise ValueError(f"out must be ({M}, {K}) (got {tuple(out.shape)})")
    _call(_dequantize, "dlrm_dequantize_int8", index,
          (q.data_ptr(), ldq, ps, M, K, out.data_ptr(), od, ldo))
    return out


def linear_int8(x_q: torch.Tensor, x_scale: torch.Tensor, w_q: torch.Tensor,
                w_scale: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none", *,
                out_dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One layer on 8-bit integers:
    ``act((x_q w_q^T) * x_scale[:, None] * w_scale + bias)``, ``(M, N)``.

    ``x_q`` ``(M, K)`` and ``w_q`` ``(N, K)`` are int8 matrices (pitch a multiple of 16),
    ``x_scale`` ``(M,)`` and ``w_scale`` ``(N,)`` f32 (one scale for each token and
    each output channel), ``bias`` ``(N,)`` f32 or None. The sum over K is exact,
    the scales are applied from left to right in f32; ``K`` is at most 131071. The
    result is f32 or bf16: ``out``, or a new tensor of ``out_dtype``. ``status`` (one
    int32) gets ``FLAG_TIMEOUT`` OR-ed in if a wait of the kernel ran out.
    """
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    M, K, ldx = _int8(x_q, "x_q", None)
    index = x_q.get_device()
    N, kw, ldw = _int8(w_q, "w_q", index)
    if kw != K:
        raise ValueError(f"w_q must be (N, {K})")
    pxs = _scales(x_scale, "x_scale", M, index)
    pws = _scales(w_scale, "w_scale", N, index)
    pb = _scales(bias, "bias", N, index) if bias is not None else None
    if out is None:
        od, ldo = ops.TABLE_DTYPES.get(out_dtype), N
        if od is None:
            raise TypeError(f"out_dtype must be float32 or bfloat16 (got {out_dtype})")
        out = _empty(M, N, out_dtype, index)
    else:
        _, od, rows, cols, ldo = _matrix(out, "out", index)
        if rows != M or cols != N:
            raise ValueError(f"out must be ({M}, {N}) (got {tuple(out.shape)})")
    # the pitch of a single row, or of none, is not used to find another: a length will do
    if M <= 1:
        ldx = (ldx + 15) // 16 * 16
    if N == 1:
        ldw = (ldw + 15) // 16 * 16
    _call(_linear, "dlrm_linear_int8", index,
          (x_q.data_ptr(), ldx, pxs, w_q.data_ptr(), ldw, pws, pb, M, N, K, code, out.data_ptr(),
           od, ldo, _status(status, index)))
    return out
