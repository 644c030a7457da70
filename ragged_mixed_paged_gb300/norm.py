"""The residual's addition and the root-mean-square norm of hidden states (``rb_add_rms_norm``)."""
from __future__ import annotations

import torch

from . import _binding as rb
from .kv4 import _device, _on, _stream, _wrong

_KINDS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_E4M3 = 3


def _rows(name: str, t, rows: int, n: int, dtype, dev: int) -> int:
    """The distance between rows of ``t`` [rows, n], whose values are adjacent."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[0] != rows or shape[1] != n or t.dtype is not dtype or \
            (stride[1] != 1 and n > 1) or t.get_device() != dev:
        _wrong(name, t, f"[{rows}, {n}] {dtype}, the values of a row adjacent", dev)
    return stride[0] if rows > 1 else n


def _norm(x, weight, eps, residual, residual_out, eight, group, out_dtype, out, scales, stream):
    if x.dim() != 2:
        raise ValueError("x must be [rows, hidden]")
    dtype = x.dtype
    kind = _KINDS.get(dtype)
    if kind is None:
        raise ValueError(f"x must be bf16, fp16 or fp32, got {dtype}")
    dev = _device("x", x)
    rows, n = x.shape
    x_stride = _rows("x", x, rows, n, dtype, dev)
    if weight.dtype is not dtype or weight.dim() != 1 or weight.shape[0] != n or \
            not weight.is_contiguous() or weight.get_device() != dev:
        _wrong("weight", weight, f"contiguous [{n}] {dtype}", dev)
    on = _stream(dev, stream)
    res_at = after_at = None
    res_stride = after_stride = 0
    if residual is not None:
        if residual_out is None:
            residual_out = residual
        res_stride = _rows("residual", residual, rows, n, dtype, dev)
        after_stride = _rows("residual_out", residual_out, rows, n, dtype, dev)
        res_at, after_at = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out without residual")
    width = n // group if group > 0 and n % group == 0 else 1
    if out is None or (eight and scales is None):
        with _on(stream):
            if out is None:
                out = torch.empty((rows, n), dtype=out_dtype or dtype, device=x.device)
            if eight and scales is None:
                scales = torch.empty((rows, width), dtype=torch.float32, device=x.device)
    _rows("out", out, rows, n, out_dtype or dtype, dev)
    if not out.is_contiguous():
        _wrong("out", out, "contiguous", dev)
    scales_at = None
    if eight:
        _rows("scales", scales, rows, width, torch.float32, dev)
        if not scales.is_contiguous():
            _wrong("scales", scales, "contiguous", dev)
        scales_at = scales.data_ptr()
    rb._check("rb_add_rms_norm", rb.lib.rb_add_rms_norm(
        rows, n, kind, x.data_ptr(), x_stride, res_at, res_stride, after_at, after_stride,
        weight.data_ptr(), eps, _E4M3 if eight else kind, group, out.data_ptr(), scales_at, on))
    return out, scales


def add_rms_norm(x, weight, eps: float = 1e-6, residual=None, residual_out=None, out=None,
                 stream=None):
    """r = x + residual, returned as r / sqrt(mean(r^2) + eps) * weight, row by row, in x's type
    (bf16, fp16 or fp32; [rows, hidden], rows any distance apart).  r goes to ``residual_out``
    (None: back into ``residual``); without a residual r is x."""
    return _norm(x, weight, eps, residual, residual_out, False, 0, None, out, None, stream)[0]


def add_rms_norm_fp8(x, weight, eps: float = 1e-6, residual=None, residual_out=None,
                     group: int = 0, out=None, scales=None, stream=None) -> tuple:
    """``add_rms_norm`` in 8 bits: (out, scales), out [rows, hidden] float8_e4m3fn whose product with
    its scale is the result; one scale a row (``group`` 0, scales [rows, 1]) or for every ``group``
    neighbouring values (16, 32, 64, 128 or 256; scales [rows, hidden / group])."""
    return _norm(x, weight, eps, residual, residual_out, True, group, torch.float8_e4m3fn, out,
                 scales, stream)
