"""This step's queries, keys and values on their way into the paged cache: rotated by their
positions (``rb_kv_append``), and a cache held in 4 bits (``rb_kv4_append``, ``rb_kv4_read``,
``rb_paged_attention_kv4``).

A cache in 4 bits is a pair of uint8 tensors [num_blocks, nkv, 9 * head_dim] (``kv4_cache``): 16 tokens
a page, a sign, two bits of exponent and one of mantissa a value, and a scale for every 16 values.
``k_scale`` and ``v_scale`` are the layer's own factors of all of them.
"""
from __future__ import annotations

import ctypes
import math
from typing import Any, Optional

import torch

from . import _binding as rb

_BF16, _I32, _U8 = torch.bfloat16, torch.int32, torch.uint8


class Rotation:
    """How positions rotate heads: ``table`` [max_position, rotary_dim] fp32 holds the cosines and
    then the sines of each position's rotary_dim / 2 angles (``rotary_table``); pair i is values
    (i, i + rotary_dim / 2) of a head, or (2i, 2i + 1) if ``interleaved``.  The table stays as it is
    (its values may change, its memory may not) while the rotation is in use."""

    def __init__(self, table, interleaved: bool = False):
        if table.dim() != 2:
            raise ValueError("table must be [max_position, rotary_dim]")
        pointer = rb._ptr(table, torch.float32, "table")
        self.table, self.interleaved = table, bool(interleaved)
        self._c = rb.rb_rotation(table.shape[1], int(self.interleaved), table.shape[0], 0, pointer)
        self._ref = ctypes.byref(self._c)


def rotary_table(max_position: int, rotary_dim: int, base: float = 10000.0, device="cuda"):
    """The table of angles p * base^(-2 i / rotary_dim), taken in 64 bits and rounded once."""
    half = torch.arange(rotary_dim // 2, dtype=torch.float64, device=device)
    angle = torch.arange(max_position, dtype=torch.float64, device=device)[:, None] * \
        base ** (-2.0 * half / rotary_dim)
    return torch.cat((torch.cos(angle), torch.sin(angle)), 1).float()


# The checks below are a good part of a small call's time: each looks for the usual case at once and
# leaves what is wrong to be named by an error path.
def _stream(dev: int, stream) -> int:
    """The stream to launch on for tensors of CUDA device ``dev``, which must be the current one."""
    if stream is None and dev == torch._C._cuda_getDevice():
        return torch._C._cuda_getCurrentRawStream(dev)
    return rb._stream_on(torch.device("cuda", dev), stream)


def _on(stream):
    return torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream())


def _device(name: str, t) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _wrong(name: str, t, what: str, dev: int):
    on = t.device
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {on}, the call's other tensors on cuda:{dev}")
    raise ValueError(f"{name} must be {what}, got {list(t.shape)} {t.dtype}, strides "
                     f"{list(t.stride())}")


def _tokens(name: str, t, heads: int, hd: int, n: int, dev: int) -> int:
    """The distance between tokens of ``t`` [n, heads, hd], whose heads and values are adjacent."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not _BF16 or len(shape) != 3 or shape[0] != n or shape[1] != heads or \
            shape[2] != hd or (stride[2] != 1 and hd > 1) or (stride[1] != hd and heads > 1) or \
            t.get_device() != dev:
        _wrong(name, t, f"bf16 [{n}, {heads}, {hd}], the heads of a token adjacent", dev)
    return stride[0] if n > 1 else heads * hd


def _int32(name: str, t, n: int, dev: int) -> int:
    if t.dtype is not _I32 or t.numel() < n or not t.is_contiguous() or t.get_device() != dev:
        _wrong(name, t, f"{n} contiguous int32", dev)
    return t.data_ptr()


def _word(error_word, dev: int) -> Optional[int]:
    return None if error_word is None else _int32("error_word", error_word, 1, dev)


def _append(call, dims, q, k, v, slot_mapping, k_cache, v_cache, positions, rotation, scales,
            q_out, error_word, stream, cache_pointer):
    nh, nkv, hd = dims.num_q_heads, dims.num_kv_heads, dims.head_dim
    dev, n = _device("k", k), k.shape[0]
    k_stride = _tokens("k", k, nkv, hd, n, dev)
    v_stride = _tokens("v", v, nkv, hd, n, dev)
    on = _stream(dev, stream)
    q_at = q_out_at = turn = position_at = None
    q_stride = q_out_stride = 0
    if q is not None:
        q_stride = _tokens("q", q, nh, hd, n, dev)
        if q_out is None:
            with _on(stream):
                q_out = torch.empty((n, nh, hd), dtype=_BF16, device=q.device)
        q_out_stride = _tokens("q_out", q_out, nh, hd, n, dev)
        q_at, q_out_at = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    if rotation is not None:
        if positions is None:
            raise ValueError("a rotation needs positions")
        if rotation.table.get_device() != dev:
            _wrong("the rotation's table", rotation.table, "", dev)
        turn, position_at = rotation._ref, _int32("positions", positions, n, dev)
    status = call(rb._dims_ref(dims), n, turn, position_at, q_at, q_stride, k.data_ptr(), k_stride,
                  v.data_ptr(), v_stride, _int32("slot_mapping", slot_mapping, n, dev), *scales,
                  q_out_at, q_out_stride, cache_pointer("k_cache", k_cache, dims, dev),
                  cache_pointer("v_cache", v_cache, dims, dev), _word(error_word, dev), on)
    if status:
        raise rb.RbError(call.__name__, status)
    return q_out


def _cache16(name: str, t, dims, dev: int) -> int:
    n = dims.num_blocks * dims.block_size * dims.num_kv_heads * dims.head_dim
    if t.dtype is not _BF16 or t.numel() < n or not t.is_contiguous() or t.get_device() != dev:
        _wrong(name, t, f"{n} contiguous bf16 values", dev)
    return t.data_ptr()


def _cache4(name: str, t, dims, dev: int) -> int:
    shape = (dims.num_blocks, dims.num_kv_heads, 9 * dims.head_dim)
    if t.dtype is not _U8 or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        _wrong(name, t, f"contiguous uint8 {list(shape)}", dev)
    return t.data_ptr()


def kv_append(dims: rb.Dims, q, k, v, slot_mapping, k_cache, v_cache, positions=None,
              rotation: Optional[Rotation] = None, q_out=None, error_word=None, stream=None):
    """Rotates ``q`` [tokens, nh, hd] and ``k`` [tokens, nkv, hd] by ``positions`` and appends k and
    ``v`` to the caches at ``slot_mapping`` (a negative slot appends nothing).  q, k and v may be
    slices of one projection's output (heads adjacent, tokens any distance apart); q may be None.
    Returns the rotated queries: ``q_out`` (q itself to rotate in place) or a new tensor."""
    return _append(rb.lib.rb_kv_append, dims, q, k, v, slot_mapping, k_cache, v_cache, positions,
                   rotation, (), q_out, error_word, stream, _cache16)


def kv4_cache(dims: rb.Dims, device="cuda") -> tuple:
    """K and V of an empty cache in 4 bits (every value 0)."""
    shape = (dims.num_blocks, dims.num_kv_heads, 9 * dims.head_dim)
    return tuple(torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2))


def kv4_page_dims(dims: rb.Dims) -> rb.Dims:
    """``dims`` with which ``PagePool`` copies and compacts whole pages of a 4-bit cache (viewed as
    ``kv4_pages``): a page is one token of 9 * head_dim / 2 values a head.  ``fork`` is for the pool of
    a 16-bit layer, whose page table both follow, or, where every layer is in 4 bits, of a stand-in
    of 16 bytes a token (1 head of 8 values); the 4-bit layers follow with ``copy``."""
    return rb.Dims(1, dims.num_q_heads, dims.num_kv_heads, 9 * dims.head_dim // 2,
                   dims.max_num_reqs, dims.max_model_len, dims.max_blocks_per_req,
                   dims.num_blocks, dims.null_block, dims.kernel_blocks_per_manager_block)


def kv4_pages(cache):
    """A 4-bit cache as the bf16 tensor that ``PagePool`` moves pages of (the same memory)."""
    return cache.view(torch.bfloat16)


def kv4_append(dims: rb.Dims, q, k, v, slot_mapping, k_cache, v_cache, positions=None,
               rotation: Optional[Rotation] = None, k_scale: float = 1.0, v_scale: float = 1.0,
               q_out=None, error_word=None, stream=None):
    """``kv_append`` into a cache held in 4 bits."""
    return _append(rb.lib.rb_kv4_append, dims, q, k, v, slot_mapping, k_cache, v_cache, positions,
                   rotation, (k_scale, v_scale), q_out, error_word, stream, _cache4)


def kv4_read(dims: rb.Dims, slots, k_cache, v_cache, k_scale: float = 1.0, v_scale: float = 1.0,
             out: Any = None, error_word=None, stream=None) -> tuple:
    """K and V rows [len(slots), nkv, hd] in bf16 of a 4-bit cache's slots (a negative slot: zeros),
    into the pair ``out`` where it is given."""
    if slots.dim() != 1:
        raise ValueError("slots must be one-dimensional")
    nkv, hd = dims.num_kv_heads, dims.head_dim
    dev, n = _device("slots", slots), slots.shape[0]
    on = _stream(dev, stream)
    if out is None:
        with _on(stream):
            out = tuple(torch.empty((n, nkv, hd), dtype=_BF16, device=slots.device)
                        for _ in range(2))
    k, v = out
    for name, t in (("out[0]", k), ("out[1]", v)):
        if _tokens(name, t, nkv, hd, n, dev) != nkv * hd:
            _wrong(name, t, "contiguous", dev)
    rb._check("rb_kv4_read", rb.lib.rb_kv4_read(
        rb._dims_ref(dims), n, _int32("slots", slots, n, dev),
        _cache4("k_cache", k_cache, dims, dev), _cache4("v_cache", v_cache, dims, dev), k_scale,
        v_scale, k.data_ptr(), v.data_ptr(), _word(error_word, dev), on))
    return k, v


def paged_attention_kv4(dims: rb.Dims, num_reqs: int, num_tokens: int, q, k_cache, v_cache,
                        block_table, query_start_loc, seq_lens, k_scale: float = 1.0,
                        v_scale: float = 1.0, out=None, workspace=None,
                        softmax_scale: Optional[float] = None, error_word=None, stream=None):
    """``paged_attention`` over a cache held in 4 bits, which holds the step's own rows already
    (``kv4_append``)."""
    nh, hd = dims.num_q_heads, dims.head_dim
    dev = _device("q", q)
    if q.dtype is not _BF16 or not q.is_contiguous() or q.dim() < 1 or \
            q.numel() != q.shape[0] * nh * hd:
        _wrong("q", q, f"contiguous bf16 [tokens, {nh}, {hd}]", dev)
    on = _stream(dev, stream)
    if out is None or workspace is None:
        with _on(stream):
            if out is None:
                out = torch.empty_like(q)
            if workspace is None:
                workspace = torch.empty(rb.workspace_size(dims, num_reqs, num_tokens), dtype=_U8,
                                        device=q.device)
    if out.dtype is not _BF16 or not out.is_contiguous() or out.numel() < q.numel() or \
            out.get_device() != dev:
        _wrong("out", out, f"{q.numel()} contiguous bf16 values", dev)
    if workspace.dtype is not _U8 or not workspace.is_contiguous() or \
            workspace.get_device() != dev:
        _wrong("workspace", workspace, "contiguous uint8", dev)
    scale = 1.0 / math.sqrt(hd) if softmax_scale is None else softmax_scale
    rb._check("rb_paged_attention_kv4", rb.lib.rb_paged_attention_kv4(
        rb._dims_ref(dims), num_reqs, num_tokens, q.shape[0], q.data_ptr(),
        _cache4("k_cache", k_cache, dims, dev), _cache4("v_cache", v_cache, dims, dev),
        _int32("block_table", block_table, num_reqs * dims.max_blocks_per_req, dev),
        _int32("query_start_loc", query_start_loc, num_reqs + 1, dev),
        _int32("seq_lens", seq_lens, num_reqs, dev), scale, k_scale, v_scale, out.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _word(error_word, dev), on))
    return out
