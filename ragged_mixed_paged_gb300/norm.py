"""The residual's addition and the root-mean-square norm of hidden states (``rb_add_rms_norm``)."""
from __future__ import annotations

from . import _binding as rb

_KINDS = {}


def _kind(t) -> int:
    import torch

    if not _KINDS:
        _KINDS.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    kind = _KINDS.get(t.dtype)
    if kind is None:
        raise ValueError(f"x must be bf16, fp16 or fp32, got {t.dtype}")
    return kind


def _rows(name: str, t, like) -> int:
    """The distance between rows of ``t``, shaped and typed as ``like``."""
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must be {list(like.shape)} {like.dtype} on {like.device}, got "
                         f"{list(t.shape)} {t.dtype} on {t.device}")
    rows, n = t.shape
    if n > 1 and t.stride(1) != 1:
        raise ValueError(f"the values of a row of {name} must be adjacent")
    return t.stride(0) if rows > 1 else n


def _norm(x, weight, eps, residual, residual_out, out_kind, group, out_dtype, out, scales, stream):
    import torch

    if x.dim() != 2 or not x.is_cuda:
        raise ValueError("x must be a CUDA tensor [rows, hidden]")
    kind = _kind(x)
    rows, n = x.shape
    device = x.device
    x_stride = _rows("x", x, x)
    if weight.shape != (n,) or weight.dtype != x.dtype or weight.device != device or \
            not weight.is_contiguous():
        raise ValueError(f"weight must be [{n}] {x.dtype} on {device}")
    on = rb._stream_on(device, stream)
    if residual is None and residual_out is not None:
        raise ValueError("residual_out without residual")
    res_at = after_at = None
    res_stride = after_stride = 0
    if residual is not None:
        if residual_out is None:
            residual_out = residual
        res_stride = _rows("residual", residual, x)
        after_stride = _rows("residual_out", residual_out, x)
        res_at, after_at = residual.data_ptr(), residual_out.data_ptr()
    eight = out_kind == 3
    width = (n // group if group and n % group == 0 else 1) if eight else 0
    if out is None or (eight and scales is None):
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            if out is None:
                out = torch.empty((rows, n), dtype=out_dtype or x.dtype, device=device)
            if eight and scales is None:
                scales = torch.empty((rows, width), dtype=torch.float32, device=device)
    if out.shape != x.shape or out.dtype != (out_dtype or x.dtype) or out.device != device or \
            not out.is_contiguous():
        raise ValueError(f"out must be contiguous {[rows, n]} {out_dtype or x.dtype} on {device}")
    if eight and (scales.shape != (rows, width) or scales.dtype != torch.float32 or
                  scales.device != device or not scales.is_contiguous()):
        raise ValueError(f"scales must be contiguous {[rows, width]} fp32 on {device}")
    rb._check("rb_add_rms_norm", rb.lib.rb_add_rms_norm(
        rows, n, kind, x.data_ptr(), x_stride, res_at, res_stride, after_at, after_stride,
        weight.data_ptr(), eps, 3 if eight else kind, group, out.data_ptr(),
        scales.data_ptr() if eight else None, on))
    return out, scales


def add_rms_norm(x, weight, eps: float = 1e-6, residual=None, residual_out=None, out=None,
                 stream=None):
    """r = x + residual, returned as r / sqrt(mean(r^2) + eps) * weight, row by row, in x's type
    (bf16, fp16 or fp32; [rows, hidden], rows any distance apart).  r goes to ``residual_out``
    (None: back into ``residual``); without a residual r is x."""
    return _norm(x, weight, eps, residual, residual_out, None, 0, None, out, None, stream)[0]


def add_rms_norm_fp8(x, weight, eps: float = 1e-6, residual=None, residual_out=None,
                     group: int = 0, out=None, scales=None, stream=None) -> tuple:
    """``add_rms_norm`` in 8 bits: (out, scales), out [rows, hidden] float8_e4m3fn whose product with
    its scale is the result; one scale a row (``group`` 0, scales [rows, 1]) or for every ``group``
    neighbouring values (16, 32, 64, 128 or 256; scales [rows, hidden / group])."""
    import torch

    return _norm(x, weight, eps, residual, residual_out, 3, group, torch.float8_e4m3fn, out,
                 scales, stream)
