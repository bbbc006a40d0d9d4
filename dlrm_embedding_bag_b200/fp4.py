"""Python binding of the 4-bit layers (the C ABI in ``include/dlrm_fp4.h``).

Argument marshalling only, as in :mod:`.optim`. A matrix in 4 bits is a pair
``(q, scale)``: uint8 ``(rows, ceil(cols / 2))``, two e2m1 codes a byte (the even
column low), with unit column stride and a row pitch that is a multiple of 16
(:func:`fp4_empty` makes such buffers), and uint8 scale tiles ``(ceil(rows / 128),
ceil(cols / 128), 512)``, one power of two (E8M0) for each 32 columns of a row in the
order that the tensor cores read.

:func:`quantize_rows` rounds activations or weights, and :func:`linear_fp4` is the
layer that multiplies the two. ``mlp.MLP(mode="fp4")`` chains them.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import ops
from .mlp import ACTS
from .optim import _call, _lib
from .tokens import (_empty, _empty_strided_cuda, _flat, _get_device, _matrix, _on, _pitch,
                     _status)

BLOCK = 32  # columns that share a scale

_quantize = _lib.dlrm_quantize_fp4
_dequantize = _lib.dlrm_dequantize_fp4
_linear = _lib.dlrm_linear_fp4


def fp4_empty(rows: int, cols: int, device="cuda") -> torch.Tensor:
    """A ``(rows, ceil(cols / 2))`` uint8 view whose row pitch is rounded up to 16."""
    width = (cols + 1) // 2
    t = torch.empty((rows, (width + 15) // 16 * 16), dtype=torch.uint8, device=device)
    return t if width % 16 == 0 else t[:, :width]


def scale_shape(rows: int, cols: int) -> Tuple[int, int, int]:
    """Shape of the scale tiles of a ``(rows, cols)`` matrix."""
    return (rows + 127) // 128, (cols + 127) // 128, 512


def _empty_tiles(rows: int, cols: int, index: int) -> torch.Tensor:
    """New scale tiles of a ``(rows, cols)`` matrix on device ``index``."""
    r, c, n = scale_shape(rows, cols)
    if _empty_strided_cuda is not None and index == _get_device():
        return _empty_strided_cuda((r, c, n), (c * n, n, 1), torch.uint8)
    return torch.empty((r, c, n), dtype=torch.uint8, device=torch.device("cuda", index))


def _codes(t: torch.Tensor, name: str, index: Optional[int]) -> Tuple[int, int, int]:
    """(rows, bytes of a row, row pitch) of a matrix of codes."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is torch.uint8) or \
            (index is not None and t.get_device() != index):
        _on(t, name, index)
        raise TypeError(f"{name} must be torch.uint8 (got {t.dtype})")
    if t.dim() == 2:  # what fp4_empty makes, without a closer look
        (rows, cols), (pitch, step) = t.shape, t.stride()
        if step == 1 and rows > 1 and pitch >= cols:
            return rows, cols, pitch
    return _pitch(t, name)


def _tiles(t: torch.Tensor, name: str, rows: int, cols: int, index: int) -> int:
    """Pointer of the scale tiles of a ``(rows, cols)`` matrix on device ``index``."""
    if isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is torch.uint8 \
            and t.is_contiguous() and t.shape == ((rows + 127) >> 7, (cols + 127) >> 7, 512):
        return t.data_ptr()
    _flat(t, name, torch.uint8, index)
    raise ValueError(f"{name} must be {scale_shape(rows, cols)} (got {tuple(t.shape)})")


def quantize_rows(x: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                  scale_out: Optional[torch.Tensor] = None):
    """``(q, scale)`` of an f32 or bf16 ``(M, K)`` matrix: for each 32 columns of a row the
    least power of two that brings the largest magnitude to 7 or less, and its elements over that
    rounded to e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6), ties to even codes. A block with a
    NaN or an infinity gets the scale NaN."""
    index, xd, M, K, ldx = _matrix(x, "x")
    width = (K + 1) // 2
    if out is None:
        ldq = (width + 15) // 16 * 16
        out = _empty(M, ldq, torch.uint8, index)
        if ldq != width:
            out = out[:, :width]
    else:
        rows, cols, ldq = _codes(out, "out", index)
        if rows != M or cols != width:
            raise ValueError(f"out must be ({M}, {width}) (got {tuple(out.shape)})")
    if scale_out is None:
        scale_out = _empty_tiles(M, K, index)
        ps = scale_out.data_ptr()
    else:
        ps = _tiles(scale_out, "scale_out", M, K, index)
    _call(_quantize, "dlrm_quantize_fp4", index,
          (x.data_ptr(), ldx, xd, M, K, out.data_ptr(), ldq, ps))
    return out, scale_out


def dequantize_rows(q: torch.Tensor, scale: torch.Tensor, cols: Optional[int] = None, *,
                    dtype: torch.dtype = torch.float32,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of a matrix in 4 bits, ``(rows, cols)``, rounded once to ``dtype``.
    ``cols`` is ``2 * q.shape[1]`` (the default) or one less."""
    M, width, ldq = _codes(q, "q", None)
    index = q.get_device()
    K = 2 * width if cols is None else cols
    if (K + 1) // 2 != width:
        raise ValueError(f"cols must be {2 * width - 1} or {2 * width} (got {cols})")
    ps = _tiles(scale, "scale", M, K, index)
    if out is None:
        od, ldo = ops.TABLE_DTYPES.get(dtype), K
        if od is None:
            raise TypeError(f"dtype must be float32 or bfloat16 (got {dtype})")
        out = _empty(M, K, dtype, index)
    else:
        _, od, rows, out_cols, ldo = _matrix(out, "out", index)
        if rows != M or out_cols != K:
            raise ValueError(f"out must be ({M}, {K}) (got {tuple(out.shape)})")
    _call(_dequantize, "dlrm_dequantize_fp4", index,
          (q.data_ptr(), ldq, ps, M, K, out.data_ptr(), od, ldo))
    return out


def linear_fp4(x_q: torch.Tensor, x_scale: torch.Tensor, w_q: torch.Tensor, w_scale: torch.Tensor,
               bias: Optional[torch.Tensor] = None, act: str = "none", *,
               out_dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One layer on 4-bit matrices: ``act(x w^T + bias)``, ``(M, N)``.

    ``(x_q, x_scale)`` is an ``(M, K)`` and ``(w_q, w_scale)`` an ``(N, K)`` matrix (pitch a
    multiple of 16; where K is odd the last half byte is zero, as
    :func:`quantize_rows` leaves it, so that rows of an odd K pass for rows of one column
    more, a zero), ``bias`` ``(N,)`` f32 or None. Products are
    exact, sums, bias and activation f32. The result is f32 or bf16: ``out``, or a new
    tensor of ``out_dtype``. ``status`` (one int32) gets ``FLAG_TIMEOUT`` OR-ed in if a
    wait of the kernel ran out.
    """
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    M, width, ldx = _codes(x_q, "x_q", None)
    index = x_q.get_device()
    N, ww, ldw = _codes(w_q, "w_q", index)
    if ww != width:
        raise ValueError(f"w_q must be (N, {width})")
    K = 2 * width
    pxs = _tiles(x_scale, "x_scale", M, K, index)
    pws = _tiles(w_scale, "w_scale", N, K, index)
    pb = None
    if bias is not None:
        pb = _flat(bias, "bias", torch.float32, index)
        if bias.numel() != N:
            raise ValueError(f"bias must have {N} elements (got {bias.numel()})")
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
    _call(_linear, "dlrm_linear_fp4", index,
          (x_q.data_ptr(), ldx, pxs, w_q.data_ptr(), ldw, pws, pb, M, N, K, code, out.data_ptr(),
           od, ldo, _status(status, index)))
    return out
