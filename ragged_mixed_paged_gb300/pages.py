"""Pages of the paged KV cache: reference counts, copies, forks, frees and compaction.

``PagePool`` binds one layer's K and V caches to a page table (for example a
``PersistentBatch``'s) and to one reference count per page, all on the device, and calls the
library's ``rb_pages_*`` kernels on them.  A "page" is what one page-table entry names.  Nothing
is synchronised; violated preconditions set bits of ``error_word`` (the ``EBIT_*`` constants).
"""
from __future__ import annotations

import ctypes

from . import _binding as rb


def pages_workspace_size(dims: rb.Dims) -> int:
    d = dims.c()
    return int(rb.lib.rb_pages_workspace_size(ctypes.byref(d)))


class PagePool:
    """One layer's caches with the page table that names their pages.

    ``block_table`` [rows, max_blocks_per_req] and ``num_blocks`` [rows] are int32 columns that
    the calls read and write in place; without them only ``copy`` works.  ``ref_count`` (int32,
    one per page) is counted from the table when it is not given.  ``batch`` takes both columns
    from a ``PersistentBatch`` and acts on its live rows; before an ``apply`` that removes rows,
    free them (their page rows are gone afterwards), and after one that adds pages, ``count``.

    What the constructor fills and counts is queued on its ``stream`` (None: the current one) and a
    call's work on the stream it is given; a caller that goes on with another stream lets that
    one wait for the first, as with any tensor.

    Further layers whose caches the same table names follow with ``copy`` on pools of their own:
    after ``fork`` from the source row's entry ``cached // page tokens`` to the new row's (-1
    where the cached tokens end at a page's end), after ``compact`` from page i to
    ``page_map[i]`` (-1 where that is -1 or i).
    """

    def __init__(self, dims: rb.Dims, k_cache, v_cache, block_table=None, num_blocks=None,
                 ref_count=None, batch=None, workspace=None, error_word=None, stream=None):
        import torch

        if batch is not None:
            if block_table is not None or num_blocks is not None:
                raise ValueError("give a batch or the table's columns, not both")
            block_table, num_blocks = batch.block_table, batch.num_blocks
        if (block_table is None) != (num_blocks is None):
            raise ValueError("block_table and num_blocks belong together")
        self.dims, self.batch = dims, batch
        self.k_cache, self.v_cache = k_cache, v_cache
        self.block_table, self.num_blocks = block_table, num_blocks
        self.device = k_cache.device
        self._i32 = torch.int32
        rows = dims.num_blocks * dims.block_size
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            if t.dim() != 3 or tuple(t.shape) != (rows, dims.num_kv_heads, dims.head_dim):
                raise ValueError(f"{name} must be [{rows}, {dims.num_kv_heads}, {dims.head_dim}]")
        self._k = rb._ptr(k_cache, torch.bfloat16, "k_cache")
        self._v = self._pointer(v_cache, torch.bfloat16, "v_cache")
        self.num_pages = dims.num_blocks // max(1, dims.kernel_blocks_per_manager_block)
        if stream is not None:
            rb._stream_on(self.device, stream)  # refuses another device's
        # what is made here is made on the stream that counts (the library clears ref_count)
        with torch.cuda.stream(stream):
            empty = lambda n, dtype: torch.empty(n, dtype=dtype, device=self.device)
            if error_word is None:
                error_word = torch.zeros(1, dtype=torch.int32, device=self.device)
            if workspace is None:
                workspace = empty(max(1, pages_workspace_size(dims)), torch.uint8)
            count = block_table is not None and ref_count is None
            if count:
                ref_count = empty(self.num_pages, torch.int32)
        self.error_word, self.workspace = error_word, workspace
        self._err = self._pointer(self.error_word, torch.int32, "error_word")
        self._ws_bytes = self.workspace.numel()
        self._ws = self._pointer(self.workspace, torch.uint8, "workspace")
        self._dims = dims.c()
        self._d = ctypes.byref(self._dims)
        self.ref_count = ref_count
        self._tables = None
        if block_table is None:
            return
        if block_table.dim() != 2 or block_table.shape[1] != dims.max_blocks_per_req:
            raise ValueError(f"block_table must be [rows, {dims.max_blocks_per_req}]")
        if num_blocks.numel() < block_table.shape[0]:
            raise ValueError("num_blocks is shorter than the block table")
        if ref_count.numel() != self.num_pages:
            raise ValueError(f"ref_count must have {self.num_pages} entries")
        i32 = torch.int32
        self._tables = rb.rb_page_tables(
            block_table.shape[0], 0, self._pointer(block_table, i32, "block_table"),
            self._pointer(num_blocks, i32, "num_blocks"),
            self._pointer(self.ref_count, i32, "ref_count"))
        if count:
            self.count(stream=stream)

    def _pointer(self, t, dtype, name):
        if t is None:
            return None
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the caches are on {self.device}")
        if t.dtype != dtype or not t.is_contiguous():
            return rb._ptr(t, dtype, name)  # names what is wrong
        return t.data_ptr()

    def _t(self):
        if self._tables is None:
            raise ValueError("this pool has no page table")
        if self.batch is not None:
            self._tables.num_rows = self.batch.num_reqs
        return ctypes.byref(self._tables)

    def _index(self, t, name):
        if t.dim() != 1:
            raise ValueError(f"{name} must have one dimension")
        return self._pointer(t, self._i32, name)

    def _one(self, t, name):
        if t is not None and t.numel() < 1:
            raise ValueError(f"{name} must hold a value")
        return self._pointer(t, self._i32, name)

    def count(self, stream=None) -> None:
        """``ref_count`` from the table: the rows that hold each page."""
        rb._check("rb_pages_count", rb.lib.rb_pages_count(
            self._d, self._t(), self._err, rb._stream_on(self.device, stream)))

    def copy(self, src, dst, stream=None) -> None:
        """K and V of page ``src[i]`` to page ``dst[i]`` (a negative id skips the pair)."""
        if src.numel() != dst.numel():
            raise ValueError("src and dst differ in length")
        rb._check("rb_pages_copy", rb.lib.rb_pages_copy(
            self._d, src.numel(), self._index(src, "src"), self._index(dst, "dst"), self._k,
            self._v, self._ws, self._ws_bytes, self._err,
            rb._stream_on(self.device, stream)))

    def fork(self, src_rows, dst_rows, num_cached, stream=None) -> None:
        """Row ``dst_rows[i]`` becomes a copy of row ``src_rows[i]`` with its
        ``num_cached[src_rows[i]]`` cached tokens: full pages shared, the partial one copied to
        the lowest free page."""
        if src_rows.numel() != dst_rows.numel():
            raise ValueError("src_rows and dst_rows differ in length")
        tables = self._t()
        if num_cached.numel() < self._tables.num_rows:
            raise ValueError("num_cached is shorter than the table")
        rb._check("rb_pages_fork", rb.lib.rb_pages_fork(
            self._d, tables, src_rows.numel(), self._index(src_rows, "src_rows"),
            self._index(dst_rows, "dst_rows"), self._index(num_cached, "num_cached"), self._k,
            self._v, self._ws, self._ws_bytes, self._err,
            rb._stream_on(self.device, stream)))

    def free(self, rows, num_freed=None, stream=None) -> None:
        """The pages of ``rows`` lose one holder each; the rows are empty afterwards."""
        rb._check("rb_pages_free", rb.lib.rb_pages_free(
            self._d, self._t(), rows.numel(), self._index(rows, "rows"),
            self._one(num_freed, "num_freed"), self._err, rb._stream_on(self.device, stream)))

    def compact(self, page_map=None, num_live=None, stream=None) -> None:
        """The live pages move to the lowest ids; ``page_map`` receives each page's new id."""
        if page_map is not None and page_map.numel() != self.num_pages:
            raise ValueError(f"page_map must have {self.num_pages} entries")
        rb._check("rb_pages_compact", rb.lib.rb_pages_compact(
            self._d, self._t(), None if page_map is None else self._index(page_map, "page_map"),
            self._one(num_live, "num_live"), self._k, self._v, self._ws,
            self._ws_bytes, self._err, rb._stream_on(self.device, stream)))
