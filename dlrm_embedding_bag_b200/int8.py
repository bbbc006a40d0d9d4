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
from .tokens import _call, _flat, _pitch, _rows, _status, _tensor

MAX_K = 131071


def int8_empty(rows: int, cols: int, device="cuda") -> torch.Tensor:
    """A ``(rows, cols)`` int8 view whose row pitch is ``cols`` rounded up to 16."""
    return torch.empty((rows, (cols + 15) // 16 * 16), dtype=torch.int8, device=device)[:, :cols]


def _int8(t: torch.Tensor, name: str, device: torch.device) -> Tuple[int, int]:
    """(pointer, row pitch) of an int8 matrix."""
    _tensor(t, name, device)
    if t.dtype != torch.int8:
        raise TypeError(f"{name} must be torch.int8 (got {t.dtype})")
    return t.data_ptr(), _pitch(t, name)


def _scales(t: torch.Tensor, name: str, n: int, device: torch.device) -> int:
    p = _flat(t, name, torch.float32, device)
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements (got {t.numel()})")
    return p


def _outputs(x, out, scale_out):
    M, K = x.shape
    if out is None:
        out = int8_empty(M, K, x.device)
    if out.shape != x.shape:
        raise ValueError(f"out must be ({M}, {K}) (got {tuple(out.shape)})")
    if scale_out is None:
        scale_out = torch.empty(M, dtype=torch.float32, device=x.device)
    pq, ldq = _int8(out, "out", x.device)
    return out, scale_out, pq, ldq, _scales(scale_out, "scale_out", M, x.device)


def quantize_rows(x: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                  scale_out: Optional[torch.Tensor] = None):
    """``(q, scale)`` of an f32 or bf16 ``(M, K)`` matrix: ``scale = max|row| / 127`` and
    ``q = row / scale`` rounded to nearest even. For weights ``(N, K)`` this is
    one scale for each output channel."""
    px, xd, ldx = _rows(x, "x")
    M, K = x.shape
    out, scale_out, pq, ldq, ps = _outputs(x, out, scale_out)
    _call("dlrm_quantize_int8", x.device, px, ldx, xd, M, K, pq, ldq, ps)
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
    px, xd, ldx = _rows(x, "x")
    M, K = x.shape
    dev = x.device
    pr, ldr, ph, ldh = None, 0, None, 0
    if residual is not None:
        if residual.dtype != x.dtype or residual.shape != x.shape:
            raise ValueError(f"residual must be {x.dtype} ({M}, {K})")
        pr, _, ldr = _rows(residual, "residual", dev)
        if residual_out is None:
            residual_out = torch.empty((M, K), dtype=x.dtype, device=dev)
        if residual_out.dtype != x.dtype or residual_out.shape != x.shape:
            raise ValueError(f"residual_out must be {x.dtype} ({M}, {K})")
        ph, _, ldh = _rows(residual_out, "residual_out", dev)
    elif residual_out is not None:
        raise ValueError("residual_out needs residual")
    pw = _scales(weight, "weight", K, dev) if weight is not None else None
    out, scale_out, pq, ldq, ps = _outputs(x, out, scale_out)
    _call("dlrm_rms_norm_int8", dev, px, ldx, pr, ldr, xd, pw, M, K, eps, ph, ldh, pq, ldq, ps)
    return out, scale_out, residual_out


def dequantize_rows(q: torch.Tensor, scale: torch.Tensor, *,
                    dtype: torch.dtype = torch.float32,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of a matrix in 8 bits, ``q * scale[:, None]``, rounded once to ``dtype``."""
    _tensor(q, "q", None)
    M, K = q.shape
    pq, ldq = _int8(q, "q", q.device)
    ps = _scales(scale, "scale", M, q.device)
    if out is None:
        out = torch.empty((M, K), dtype=dtype, device=q.device)
    if out.shape != q.shape:
        raise ValueError(f"out must be ({M}, {K}) (got {tuple(out.shape)})")
    po, od, ldo = _rows(out, "out", q.device)
    _call("dlrm_dequantize_int8", q.device, pq, ldq, ps, M, K, po, od, ldo)
    return out


def linear_int8(x_q: torch.Tensor, x_scale: torch.Tensor, w_q: torch.Tensor,
                w_scale: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none", *,
                out_dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One layer on 8-bit integers:
    ``act((x_q w_q^T) * x_scale[:, None] * w_scale + bias)``, ``(M, N)``.

    ``x_q`` ``(M, K)`` and ``w_q`` ``(N, K)`` are int8 matrices (pitch a multiple of 16),
    ``x_scale`` ``(M,)`` and ``w_scale`` ``(N,)`` f32 (one scale for each token and
    each output channel), ``bias`` ``(N,)`` f32 or None. The sum over K is exact;
    ``K`` is at most 131071. The result is f32 or bf16 (``out_dtype``).
    """
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    _tensor(x_q, "x_q", None)
    dev = x_q.device
    px, ldx = _int8(x_q, "x_q", dev)
    pw, ldw = _int8(w_q, "w_q", dev)
    M, K = x_q.shape
    N = w_q.shape[0]
    if w_q.shape[1] != K:
        raise ValueError(f"w_q must be (N, {K})")
    pxs = _scales(x_scale, "x_scale", M, dev)
    pws = _scales(w_scale, "w_scale", N, dev)
    pb = _scales(bias, "bias", N, dev) if bias is not None else None
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out must be ({M}, {N}) (got {tuple(out.shape)})")
    po, od, ldo = _rows(out, "out", dev)
    # a single row's pitch is not used to find another one: its own length will do
    if M == 1:
        ldx = (ldx + 15) // 16 * 16
    if N == 1:
        ldw = (ldw + 15) // 16 * 16
    _call("dlrm_linear_int8", dev, px, ldx, pxs, pw, ldw, pws, pb, M, N, K, ACTS[act], po, od, ldo,
          _status(status, dev))
    return out
