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

`stream` gives a call to another stream than the current one.  What it allocates comes from that stream's memory; that
the cache and the tensors it is given are ready there is the caller's to see to.
"""
from __future__ import annotations

import dataclasses
import math
from typing import Optional, Tuple

import torch

from . import WQError, _check_cuda, _check_tensor, _dt, _empty, _need, _ptr, _stream, lib


@dataclasses.dataclass(frozen=True)
class KVCache:
    """The cache of one layer: the library's buffer plus its description."""
    data: torch.Tensor      # uint8 device buffer of wq_kv_cache_bytes()
    num_pages: int
    page_size: int
    kv_heads: int
    head_dim: int
    group: int
    dtype: torch.dtype      # type of the rows written: float16 or bfloat16

    def __post_init__(self):
        for name in ("num_pages", "page_size", "kv_heads", "head_dim", "group"):
            v = getattr(self, name)
            _need(isinstance(v, int) and 0 < v < 1 << 31, f"{name} must be a positive 32-bit count, got {v!r}")
        nbytes = wq_kv_cache_bytes(self.num_pages, self.page_size, self.kv_heads, self.head_dim, self.group)
        _need(nbytes > 0, "the cache's description is not one the library supports")
        object.__setattr__(self, "nbytes", nbytes)
        object.__setattr__(self, "dt", _dt(self.dtype))


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


# The checks below run on every call, so the common case takes one chain of
# comparisons; what is wrong is named only after it failed.
def _check_cache(cache: KVCache) -> torch.Tensor:
    d = cache.data
    if not (isinstance(d, torch.Tensor) and d.dtype == torch.uint8 and d.dim() == 1 and d.is_contiguous()):
        raise ValueError("cache.data must be a contiguous 1-D uint8 tensor")
    if d.numel() < cache.nbytes:
        raise ValueError("cache.data is shorter than the cache it describes")
    return d


def _check_rows(x, name: str, cache: KVCache, dev, heads: Optional[int], rows: Optional[int]) -> Tuple[int, int]:
    """x [rows][heads][head_dim] of the cache's type on `dev`; rows may be strided, a row is contiguous.  Returns the
    address and the elements between rows."""
    if isinstance(x, torch.Tensor) and x.dim() == 3:
        n, h, d = x.shape
        sn, sh, sd = x.stride()
        at = x.data_ptr()
        if n <= 1:
            sn = h * d
        if (d == cache.head_dim and x.dtype == cache.dtype and (rows is None or n == rows)
                and (heads is None or h == heads) and x.device == dev
                and (n == 0 or h == 0 or (sd == 1 and (h == 1 or sh == d) and sn >= h * d and sn % 8 == 0
                                          and at % 16 == 0))):
            return at, sn
    _need(isinstance(x, torch.Tensor) and x.dim() == 3, f"{name} must be a [rows][heads][head_dim] tensor")
    _need(x.dtype == cache.dtype, f"{name} must have the cache's dtype {cache.dtype}, got {x.dtype}")
    _need(d == cache.head_dim, f"{name} must have head_dim {cache.head_dim}, got {d}")
    _need(heads is None or h == heads, f"{name} must have {heads} heads, got {h}")
    _need(rows is None or n == rows, f"{name} must have {rows} rows, got {n}")
    _need(x.device == dev, f"{name} and the cache must be on the same device")
    _need(sd == 1 and (h == 1 or sh == d), f"the heads of a row of {name} must be contiguous")
    _need(sn >= h * d and sn % 8 == 0, f"the row stride of {name} must be a multiple of 8 elements and hold a row")
    raise ValueError(f"{name} must be 16-byte aligned")


def _check_seqs(dev, block_table, kv_lens, cu_q, rows: int) -> Tuple[int, int]:
    if not (isinstance(block_table, torch.Tensor) and block_table.dim() == 2):
        raise ValueError("block_table must be a [batch][pages] tensor")
    batch, max_pages = block_table.shape
    if not (block_table.dtype == torch.int32 and block_table.is_contiguous() and block_table.device == dev
            and isinstance(kv_lens, torch.Tensor) and kv_lens.dtype == torch.int32 and kv_lens.shape == (batch,)
            and kv_lens.is_contiguous() and kv_lens.device == dev):
        _check_tensor(block_table, "block_table", (torch.int32,), (batch, max_pages), dev)
        _check_tensor(kv_lens, "kv_lens", (torch.int32,), (batch,), dev)
    if cu_q is not None:
        _check_tensor(cu_q, "cu_q", (torch.int32,), (batch + 1,), dev)
    elif rows and (batch == 0 or rows % batch):
        raise ValueError(f"without cu_q every sequence has as many rows: {rows} rows of {batch} sequences")
    if rows and batch == 0:
        raise ValueError("rows need a sequence")
    return batch, max_pages


def wq_kv_write(k: torch.Tensor, v: torch.Tensor, cache: KVCache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                cu_q: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantise the rows k, v [rows][kv_heads][head_dim] into the cache (their heads contiguous, rows strided at
    will: slices of a fused projection's output are fine)."""
    data = _check_cache(cache)
    dev = data.device
    k_at, ld_k = _check_rows(k, "k", cache, dev, cache.kv_heads, None)
    rows = k.shape[0]
    v_at, ld_v = _check_rows(v, "v", cache, dev, cache.kv_heads, rows)
    batch, max_pages = _check_seqs(dev, block_table, kv_lens, cu_q, rows)
    _check_cuda(data, "cache.data")
    rc = lib().wq_kv_write(k_at, v_at, ld_k, ld_v, cache.dt, data.data_ptr(), block_table.data_ptr(),
                           kv_lens.data_ptr(), _ptr(cu_q), rows, batch, max_pages, cache.num_pages, cache.page_size,
                           cache.kv_heads, cache.head_dim, cache.group, _stream(stream, dev))
    if rc:
        raise WQError("wq_kv_write", rc)


def wq_kv_read(cache: KVCache, block_table: torch.Tensor, kv_lens: torch.Tensor, rows: int,
               cu_q: Optional[torch.Tensor] = None, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The cached keys and values of the rows' places, each [rows][kv_heads][head_dim] in the cache's type.  Rows
    outside every sequence of cu_q are left as they were in `out` (undefined where this call allocates it)."""
    data = _check_cache(cache)
    dev = data.device
    if not (isinstance(rows, int) and rows >= 0):
        raise ValueError("rows must be a count")
    batch, max_pages = _check_seqs(dev, block_table, kv_lens, cu_q, rows)
    if out is not None:
        k, v = out
        k_at, ld_k = _check_rows(k, "out[0]", cache, dev, cache.kv_heads, rows)
        v_at, ld_v = _check_rows(v, "out[1]", cache, dev, cache.kv_heads, rows)
    _check_cuda(data, "cache.data")
    at = _stream(stream, dev)
    if out is None:
        k, v = (_empty(stream, data, (rows, cache.kv_heads, cache.head_dim), cache.dtype) for _ in range(2))
        k_at, v_at, ld_k = k.data_ptr(), v.data_ptr(), cache.kv_heads * cache.head_dim
        ld_v = ld_k
    rc = lib().wq_kv_read(data.data_ptr(), k_at, v_at, ld_k, ld_v, cache.dt, block_table.data_ptr(),
                          kv_lens.data_ptr(), _ptr(cu_q), rows, batch, max_pages, cache.num_pages, cache.page_size,
                          cache.kv_heads, cache.head_dim, cache.group, at)
    if rc:
        raise WQError("wq_kv_read", rc)
    return k, v


def wq_kv_workspace_bytes(rows: int, batch: int, ragged: bool, q_heads: int, kv_heads: int, head_dim: int,
                          group: int, max_kv_len: int) -> int:
    """Scratch of a wq_kv_attention call with these sizes (ragged: with cu_q; max_kv_len: past 2^30 as 2^30, as that
    call takes it).  Fewer rows may need more of it: ask for every shape that is used."""
    return int(lib().wq_kv_workspace_bytes(rows, batch, int(bool(ragged)), q_heads, kv_heads, head_dim, group,
                                           min(max_kv_len, 1 << 30)))


def wq_kv_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                    cu_q: Optional[torch.Tensor] = None, scale: Optional[float] = None, causal: bool = True,
                    window: int = 0, max_kv_len: Optional[int] = None, out: Optional[torch.Tensor] = None, ws=None,
                    stream=None) -> torch.Tensor:
    """softmax(scale q K^T) V over the cache; q [rows][q_heads][head_dim], q_heads a multiple of the cache's heads.

    scale: head_dim ** -0.5 by default.  causal: a row sees the positions up to its own.  window > 0: only the last
    `window` of them.  max_kv_len: the longest length to expect (the table's capacity by default); it only shapes the
    launch.  ws: wq_kv_workspace_bytes() bytes of scratch, allocated when not given.  Rows outside every sequence of
    cu_q are left as they were in `out` (undefined where this call allocates it)."""
    data = _check_cache(cache)
    dev = data.device
    q_at, ld_q = _check_rows(q, "q", cache, dev, None, None)
    rows, q_heads = q.shape[0], q.shape[1]
    if q_heads == 0 or q_heads % cache.kv_heads:
        raise ValueError(f"q must have a multiple of the cache's {cache.kv_heads} heads, got {q_heads}")
    batch, max_pages = _check_seqs(dev, block_table, kv_lens, cu_q, rows)
    if scale is None:
        scale = cache.head_dim ** -0.5
    elif not (scale > 0 and math.isfinite(scale)):
        raise ValueError(f"scale must be positive and finite, got {scale}")
    if not (isinstance(window, int) and window >= 0):
        raise ValueError(f"window must be 0 or a count, got {window}")
    if window > 1 << 30:  # no position lies that far back
        window = 1 << 30
    if max_kv_len is None:
        max_kv_len = max_pages * cache.page_size
    elif not (isinstance(max_kv_len, int) and max_kv_len >= 0):
        raise ValueError("max_kv_len must be a count")
    if max_kv_len > 1 << 30:
        max_kv_len = 1 << 30
    L = lib()
    need = L.wq_kv_workspace_bytes(rows, batch, cu_q is not None, q_heads, cache.kv_heads, cache.head_dim,
                                   cache.group, max_kv_len)
    if ws is not None and need:
        _need(isinstance(ws, torch.Tensor) and ws.is_contiguous() and ws.device == dev,
              "ws must be a contiguous tensor on the device of q")
        _need(ws.numel() * ws.element_size() >= need, lambda: f"ws holds fewer than the {need} bytes this call needs")
    if out is not None:
        o_at, ld_o = _check_rows(out, "out", cache, dev, q_heads, rows)
    _check_cuda(data, "cache.data")
    at = _stream(stream, dev)
    if out is None:
        out = _empty(stream, q, (rows, q_heads, cache.head_dim))
        o_at, ld_o = out.data_ptr(), q_heads * cache.head_dim
    if need and ws is None:
        ws = _empty(stream, data, need, scratch=True)
    rc = L.wq_kv_attention(q_at, ld_q, cache.dt, data.data_ptr(), block_table.data_ptr(), kv_lens.data_ptr(),
                           _ptr(cu_q), o_at, ld_o, rows, batch, max_pages, cache.num_pages, cache.page_size, q_heads,
                           cache.kv_heads, cache.head_dim, cache.group, scale, 1 if causal else 0, window, max_kv_len,
                           ws.data_ptr() if need else None, need, at)
    if rc:
        raise WQError("wq_kv_attention", rc)
    return out
