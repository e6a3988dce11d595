"""Page tables of the 4-bit cache, kept on the GPU: lengths, block table and free pages of a batch of sequences.

Like the rest of the package this only checks and marshals arguments (rules: include/wq.h).  A step of a serving loop
names the lengths its sequences shall have, and gets the offsets and positions of the new rows that every other call
takes; nothing comes back to the host, so the whole step can be captured:

    cu_q, positions, _ = wq.wq_kv_resize(pages, lens, rows)
    y = stack.step(x, pages.block_table, pages.kv_lens, cu_q)
"""
from __future__ import annotations

import dataclasses
from typing import Optional, Tuple

import torch

from . import WQError, _check_cuda, _check_tensor, _empty, _need, _ptr, _stream, lib


@dataclasses.dataclass(frozen=True)
class KVPages:
    """Which pages the sequences of a batch hold; one description serves the caches of all layers."""
    block_table: torch.Tensor  # int32 [batch][max_pages]
    kv_lens: torch.Tensor      # int32 [batch]
    free: torch.Tensor         # int32 [num_pages]: a stack of free pages, the next one to be taken on top
    counts: torch.Tensor       # int32 [2]: free pages; what the last change lacked (0: done, -1: not a change)
    num_pages: int
    page_size: int

    def __post_init__(self):
        _need(isinstance(self.block_table, torch.Tensor) and self.block_table.dim() == 2,
              "block_table must be a [batch][pages] tensor")
        dev, (batch, _) = self.block_table.device, self.block_table.shape
        _need(isinstance(self.num_pages, int) and 0 < self.num_pages <= 1 << 30,
              "num_pages must be a positive count up to 2^30")
        _need(isinstance(self.page_size, int) and 16 <= self.page_size <= 1024
              and self.page_size & (self.page_size - 1) == 0, "page_size must be a power of two from 16 to 1024")
        _check_tensor(self.block_table, "block_table", (torch.int32,), self.block_table.shape)
        _check_tensor(self.kv_lens, "kv_lens", (torch.int32,), (batch,), dev)
        _check_tensor(self.free, "free", (torch.int32,), (self.num_pages,), dev)
        _check_tensor(self.counts, "counts", (torch.int32,), (2,), dev)


def wq_kv_pages(num_pages: int, page_size: int, batch: int, max_pages: int, device="cuda") -> KVPages:
    """`num_pages` free pages and `batch` empty sequences of at most `max_pages` pages each."""
    _need(isinstance(num_pages, int) and 0 < num_pages <= 1 << 30, "num_pages must be a positive count up to 2^30")
    i32 = dict(dtype=torch.int32, device=device)
    return KVPages(torch.full((batch, max_pages), -1, **i32), torch.zeros(batch, **i32),
                   torch.arange(num_pages - 1, -1, -1, **i32), torch.tensor([num_pages, 0], **i32), num_pages, page_size)


def wq_kv_resize_workspace_bytes(batch: int, max_pages: int, num_pages: int, rows: int) -> int:
    """Scratch of a wq_kv_resize call with these sizes."""
    return int(lib().wq_kv_resize_workspace_bytes(batch, max_pages, num_pages, rows))


def wq_kv_resize(pages: KVPages, want_lens: torch.Tensor, rows: int = 0, cu_q: Optional[torch.Tensor] = None,
                 positions: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None, ws=None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The sequences of `pages` become want_lens (int32 [batch]) tokens long: pages are taken or given back, kv_lens,
    the table, the free pages and counts are changed in place -- or, where the free pages do not suffice, a length has no
    place in the table or the new tokens are more than 2^31 - 1 in all, nothing is but counts[1] (the pages lacking, or
    -1; 0 where all went well).

    Returns (cu_q, positions, slots): int32 [batch + 1] offsets of the new rows (all 0 where nothing was changed),
    int32 [rows] position and int64 [rows] slot (page * page_size + place in it) of each; `rows` is how many the
    program makes room for, entries past the new rows are -1.  They go to the given tensors, or to new ones.  ws:
    wq_kv_resize_workspace_bytes() bytes of scratch, allocated when not given."""
    table = pages.block_table
    dev, (batch, max_pages) = table.device, table.shape
    if not (isinstance(rows, int) and rows >= 0):
        raise ValueError("rows must be a count")
    if not (isinstance(want_lens, torch.Tensor) and want_lens.dtype == torch.int32 and want_lens.shape == (batch,)
            and want_lens.is_contiguous() and want_lens.device == dev):
        _check_tensor(want_lens, "want_lens", (torch.int32,), (batch,), dev)
    for t, name, dtype, n in ((cu_q, "cu_q", torch.int32, batch + 1), (positions, "positions", torch.int32, rows),
                              (slots, "slots", torch.int64, rows)):
        if t is not None:
            _check_tensor(t, name, (dtype,), (n,), dev)
    L = lib()
    need = L.wq_kv_resize_workspace_bytes(batch, max_pages, pages.num_pages, rows)
    if ws is not None and need:
        _need(isinstance(ws, torch.Tensor) and ws.is_contiguous() and ws.device == dev,
              "ws must be a contiguous tensor on the device of the pages")
        _need(ws.numel() * ws.element_size() >= need, lambda: f"ws holds fewer than the {need} bytes this call needs")
    _check_cuda(table, "pages.block_table")
    at = _stream(stream, dev)
    if cu_q is None:
        cu_q = _empty(stream, table, (batch + 1,))
    if positions is None:
        positions = _empty(stream, table, (rows,))
    if slots is None:
        slots = _empty(stream, table, (rows,), torch.int64)
    if need and ws is None:
        ws = _empty(stream, table, need, torch.uint8, scratch=True)
    rc = L.wq_kv_resize(table.data_ptr(), pages.kv_lens.data_ptr(), want_lens.data_ptr(), pages.free.data_ptr(),
                        pages.counts.data_ptr(), cu_q.data_ptr(), positions.data_ptr() if rows else None,
                        slots.data_ptr() if rows else None, rows, batch, max_pages, pages.num_pages, pages.page_size,
                        ws.data_ptr() if need else None, need, at)
    if rc:
        raise WQError("wq_kv_resize", rc)
    return cu_q, positions, slots
