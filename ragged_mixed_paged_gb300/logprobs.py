"""Log probabilities of given tokens, with entropy and top alternatives (``rb_token_logprobs``)."""
from __future__ import annotations

from dataclasses import dataclass
from typing import Any

from . import _binding as rb

MAX_TOP_LOGPROBS = 32


@dataclass
class TokenLogprobs:
    """Results of ``token_logprobs``, one entry per row of logits (natural logarithms)."""

    logprobs: Any       # [rows] fp32, of the given token
    ranks: Any          # [rows] int32, 1 + the number of larger logits
    entropy: Any        # [rows] fp32
    top_ids: Any        # [rows, top_k] int32, largest logit first, ties by id
    top_logprobs: Any   # [rows, top_k] fp32

    @classmethod
    def allocate(cls, rows: int, top_k: int, device="cuda") -> "TokenLogprobs":
        import torch

        f32, i32 = torch.float32, torch.int32
        new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=device)
        return cls(new(rows, f32), new(rows, i32), new(rows, f32), new((rows, top_k), i32),
                   new((rows, top_k), f32))


def token_logprobs(logits, token_ids, top_k: int = 0, out: TokenLogprobs = None,
                   error_word=None, stream=None) -> TokenLogprobs:
    """Log probability and rank of ``token_ids[r]`` in row r of ``logits`` [rows, vocab] (bf16,
    fp16 or fp32; a row's elements adjacent, rows any distance of at least ``vocab`` apart), the
    row's entropy, and its ``top_k`` (at most 32) most likely tokens.  A token id of -1 asks
    for none (log probability 0, rank 0)."""
    import torch

    if logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor [rows, vocab]")
    f32, i32 = torch.float32, torch.int32
    kind = {torch.bfloat16: 0, torch.float16: 1, f32: 2}.get(logits.dtype)
    if kind is None:
        raise ValueError(f"logits must be bf16, fp16 or fp32, got {logits.dtype}")
    device = logits.device
    rows, vocab = logits.shape
    stride = logits.stride(0) if rows > 1 else vocab
    if vocab > 1 and logits.stride(1) != 1:
        raise ValueError("the elements of a row of logits must be adjacent")
    if stride < vocab:
        raise ValueError("rows of logits must not overlap")
    if token_ids.shape != (rows,):
        raise ValueError(f"token_ids must be [{rows}]")
    if out is None:
        s = stream if stream is not None else torch.cuda.current_stream(logits.device)
        with torch.cuda.stream(s):
            out = TokenLogprobs.allocate(rows, top_k, logits.device)
    pointers = []
    for name, dtype, shape in (("logprobs", f32, (rows,)), ("ranks", i32, (rows,)),
                               ("entropy", f32, (rows,)), ("top_ids", i32, (rows, top_k)),
                               ("top_logprobs", f32, (rows, top_k))):
        t = getattr(out, name)
        if t.shape != shape:
            raise ValueError(f"out.{name} must be {list(shape)}")
        if t.device != device:
            raise ValueError(f"out.{name} is on {t.device}, the logits are on {device}")
        if t.dtype != dtype or not t.is_contiguous():
            rb._ptr(t, dtype, f"out.{name}")  # names what is wrong
        pointers.append(t.data_ptr())
    for name, t in (("token_ids", token_ids), ("error_word", error_word)):
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the logits are on {device}")
    rb._check("rb_token_logprobs", rb.lib.rb_token_logprobs(
        rows, vocab, stride, kind, logits.data_ptr(),
        rb._ptr(token_ids, i32, "token_ids"), top_k, *pointers,
        rb._ptr(error_word, i32, "error_word"), rb._stream_on(device, stream)))
    return out
