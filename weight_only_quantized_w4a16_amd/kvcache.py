"""4-bit paged key/value cache: rows quantised as they are written, read back,
and attention over the codes.

Like the rest of the package these functions only check and marshal arguments;
every step runs in the library's kernels (layout and arithmetic: include/wq.h).
All of them name rows and sequences the same way:

  block_table  int32 [batch][max_pages]: page of positions page_size * p ...
  kv_lens      int32 [batch]: length of each sequence, the call's rows included
  cu_q         int32 [batch + 1]: first row of each sequence, ascending; None:
               rows / batch rows each (one each in a decode step)

so the rows of sequence b are its last cu_q[b + 1] - cu_q[b] positions.
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
from typing import Optional, Tuple

import torch

from . import _check, _check_cuda, _check_tensor, _dt, _need, _ptr, _stream, WQError, lib


@dataclasses.dataclass
class KVCache:
    """The cache of one layer: the library's buffer plus its description."""
    data: torch.Tensor      # uint8 device buffer of wq_kv_cache_bytes()
    num_pages: int
    page_size: int
    kv_heads: int
    head_dim: int
    group: int
    dtype: torch.dtype      # type of the rows written: float16 or bfloat16


def wq_kv_cache_bytes(num_pages: int, page_size: int, kv_heads: int, head_dim: int, group: int) -> int:
    return int(lib().wq_kv_cache_bytes(num_pages, page_size, kv_heads, head_dim, group))


def wq_kv_cache(num_pages: int, page_size: int, kv_heads: int, head_dim: int, group: int = 128,
                dtype: torch.dtype = torch.float16, device="cuda") -> KVCache:
    """An uninitialised cache of `num_pages` pages (head_dim 64, 96, 128, 192 or 256;
    group 32, 64 or 128; page_size a power of two from 16 to 1024)."""
    _dt(dtype)
    nbytes = wq_kv_cache_bytes(num_pages, page_size, kv_heads, head_dim, group)
    if nbytes == 0:
        raise WQError("wq_kv_cache_bytes", 2)
    return KVCache(torch.empty(nbytes, dtype=torch.uint8, device=device), num_pages, page_size, kv_heads, head_dim,
                   group, dtype)


def _check_cache(cache: KVCache):
    d = cache.data
    _need(isinstance(d, torch.Tensor) and d.dtype == torch.uint8 and d.dim() == 1 and d.is_contiguous(),
          "cache.data must be a contiguous 1-D uint8 tensor")
    need = wq_kv_cache_bytes(cache.num_pages, cache.page_size, cache.kv_heads, cache.head_dim, cache.group)
    _need(need > 0, "the cache's description is not one the library supports")
    _need(d.numel() >= need, "cache.data is shorter than the cache it describes")


def _check_rows(x, name: str, cache: KVCache, heads: Optional[int], rows: Optional[int]):
    """x [rows][heads][head_dim] of the cache's type; rows may be strided, a row is contiguous."""
    _need(isinstance(x, torch.Tensor) and x.dim() == 3, lambda: f"{name} must be a [rows][heads][head_dim] tensor")
    _need(x.dtype == cache.dtype, lambda: f"{name} must have the cache's dtype {cache.dtype}, got {x.dtype}")
    _need(x.shape[2] == cache.head_dim, lambda: f"{name} must have head_dim {cache.head_dim}, got {x.shape[2]}")
    _need(heads is None or x.shape[1] == heads, lambda: f"{name} must have {heads} heads, got {x.shape[1]}")
    _need(rows is None or x.shape[0] == rows, lambda: f"{name} must have {rows} rows, got {x.shape[0]}")
    _need(x.numel() == 0 or (x.stride(2) == 1 and (x.shape[1] == 1 or x.stride(1) == cache.head_dim)),
          lambda: f"the heads of a row of {name} must be contiguous")
    _need(x.shape[0] <= 1 or (x.stride(0) >= x.shape[1] * x.shape[2] and x.stride(0) % 8 == 0),
          lambda: f"the row stride of {name} must be a multiple of 8 elements and hold a row")
    _need(x.numel() == 0 or x.data_ptr() % 16 == 0, lambda: f"{name} must be 16-byte aligned")
    _need(x.device == cache.data.device, lambda: f"{name} and the cache must be on the same device")


def _check_seqs(cache: KVCache, block_table, kv_lens, cu_q, rows: int) -> Tuple[int, int]:
    dev = cache.data.device
    _need(isinstance(block_table, torch.Tensor) and block_table.dim() == 2, "block_table must be a [batch][pages] tensor")
    batch, max_pages = block_table.shape
    _check_tensor(block_table, "block_table", (torch.int32,), (batch, max_pages), dev)
    _check_tensor(kv_lens, "kv_lens", (torch.int32,), (batch,), dev)
    if cu_q is not None:
        _check_tensor(cu_q, "cu_q", (torch.int32,), (batch + 1,), dev)
    else:
        _need(rows == 0 or (batch > 0 and rows % batch == 0),
              lambda: f"without cu_q every sequence has as many rows: {rows} rows of {batch} sequences")
    _need(rows == 0 or batch > 0, "rows need a sequence")
    return batch, max_pages


def _ld(x: torch.Tensor) -> int:
    return x.stride(0) if x.shape[0] > 1 else x.shape[1] * x.shape[2]


def _shape_args(cache: KVCache, rows: int, batch: int, max_pages: int):
    return rows, batch, max_pages, cache.num_pages, cache.page_size


def wq_kv_write(k: torch.Tensor, v: torch.Tensor, cache: KVCache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                cu_q: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantise the rows k, v [rows][kv_heads][head_dim] into the cache (their heads contiguous, rows strided at
    will: slices of a fused projection's output are fine)."""
    _check_cache(cache)
    _check_rows(k, "k", cache, cache.kv_heads, None)
    _check_rows(v, "v", cache, cache.kv_heads, k.shape[0])
    rows = k.shape[0]
    batch, max_pages = _check_seqs(cache, block_table, kv_lens, cu_q, rows)
    _check_cuda(k, "k")
    rc = lib().wq_kv_write(_ptr(k), _ptr(v), _ld(k), _ld(v), _dt(cache.dtype), _ptr(cache.data), _ptr(block_table),
                           _ptr(kv_lens), _ptr(cu_q), *_shape_args(cache, rows, batch, max_pages), cache.kv_heads,
                           cache.head_dim, cache.group, _stream(stream, k.device))
    _check("wq_kv_write", rc)


def wq_kv_read(cache: KVCache, block_table: torch.Tensor, kv_lens: torch.Tensor, rows: int,
               cu_q: Optional[torch.Tensor] = None, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The cached keys and values of the rows' places, each [rows][kv_heads][head_dim] in the cache's type.  Rows
    outside every sequence of cu_q are left as they were in `out` (undefined where this call allocates it)."""
    _check_cache(cache)
    _need(isinstance(rows, int) and rows >= 0, "rows must be a count")
    batch, max_pages = _check_seqs(cache, block_table, kv_lens, cu_q, rows)
    shape, dev = (rows, cache.kv_heads, cache.head_dim), cache.data.device
    if out is None:
        k, v = (torch.empty(shape, dtype=cache.dtype, device=dev) for _ in range(2))
    else:
        k, v = out
        _check_rows(k, "out[0]", cache, cache.kv_heads, rows)
        _check_rows(v, "out[1]", cache, cache.kv_heads, rows)
    _check_cuda(cache.data, "cache.data")
    rc = lib().wq_kv_read(_ptr(cache.data), _ptr(k), _ptr(v), _ld(k), _ld(v), _dt(cache.dtype), _ptr(block_table),
                          _ptr(kv_lens), _ptr(cu_q), *_shape_args(cache, rows, batch, max_pages), cache.kv_heads,
                          cache.head_dim, cache.group, _stream(stream, dev))
    _check("wq_kv_read", rc)
    return k, v


def wq_kv_workspace_bytes(rows: int, batch: int, ragged: bool, q_heads: int, kv_heads: int, head_dim: int,
                          group: int, max_kv_len: int) -> int:
    return int(lib().wq_kv_workspace_bytes(rows, batch, int(bool(ragged)), q_heads, kv_heads, head_dim, group,
                                           max_kv_len))


def wq_kv_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                    cu_q: Optional[torch.Tensor] = None, scale: Optional[float] = None, causal: bool = True,
                    window: int = 0, max_kv_len: Optional[int] = None, out: Optional[torch.Tensor] = None, ws=None,
                    stream=None) -> torch.Tensor:
    """softmax(scale q K^T) V over the cache; q [rows][q_heads][head_dim], q_heads a multiple of the cache's heads.

    scale: head_dim ** -0.5 by default.  causal: a row sees the positions up to its own.  window > 0: only the last
    `window` of them.  max_kv_len: the longest length to expect (the table's capacity by default); it only shapes the
    launch.  ws: wq_kv_workspace_bytes() bytes of scratch, allocated when not given.  Rows outside every sequence of
    cu_q are left as they were in `out` (undefined where this call allocates it)."""
    _check_cache(cache)
    _check_rows(q, "q", cache, None, None)
    rows, q_heads = q.shape[0], q.shape[1]
    _need(q_heads > 0 and q_heads % cache.kv_heads == 0,
          lambda: f"q must have a multiple of the cache's {cache.kv_heads} heads, got {q_heads}")
    batch, max_pages = _check_seqs(cache, block_table, kv_lens, cu_q, rows)
    if scale is None:
        scale = cache.head_dim ** -0.5
    _need(scale > 0 and math.isfinite(scale), lambda: f"scale must be positive and finite, got {scale}")
    _need(isinstance(window, int) and window >= 0, lambda: f"window must be 0 or a count, got {window}")
    if max_kv_len is None:
        max_kv_len = max_pages * cache.page_size
    _need(isinstance(max_kv_len, int) and max_kv_len >= 0, "max_kv_len must be a count")
    if out is not None:
        _check_rows(out, "out", cache, q_heads, rows)
    need = wq_kv_workspace_bytes(rows, batch, cu_q is not None, q_heads, cache.kv_heads, cache.head_dim,
                                 cache.group, max_kv_len)
    if ws is not None and need:
        _need(isinstance(ws, torch.Tensor) and ws.is_contiguous() and ws.device == q.device,
              "ws must be a contiguous tensor on the device of q")
        _need(ws.numel() * ws.element_size() >= need, lambda: f"ws holds fewer than the {need} bytes this call needs")
    _check_cuda(q, "q")
    if out is None:
        out = torch.empty((rows, q_heads, cache.head_dim), dtype=q.dtype, device=q.device)
    if need and ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    rc = lib().wq_kv_attention(_ptr(q), _ld(q), _dt(cache.dtype), _ptr(cache.data), _ptr(block_table), _ptr(kv_lens),
                               _ptr(cu_q), _ptr(out), _ld(out), *_shape_args(cache, rows, batch, max_pages), q_heads,
                               cache.kv_heads, cache.head_dim, cache.group, ctypes.c_float(scale), int(bool(causal)),
                               window, max_kv_len, _ptr(ws) if need else None, need if need else 0,
                               _stream(stream, q.device))
    _check("wq_kv_attention", rc)
    return out
