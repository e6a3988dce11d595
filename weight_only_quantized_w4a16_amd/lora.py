"""Low-rank adapters of many sequences beside one shared (quantised) projection.

Like the rest of the package this only checks and marshals arguments (arithmetic: include/wq.h).  A bank holds the
adapters of one projection; each sequence of a call names its own, so that requests of many fine-tuned variants share
the packed weights:

    y = wq.linear(x, layer, bias=b)
    wq.wq_lora(x, bank, adapters, y, cu_q=cu_q, out=y)
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional, Tuple

import torch

from . import WQError, _check_cuda, _check_tensor, _dt, _empty, _need, _ptr, _stream, lib


@dataclasses.dataclass(frozen=True)
class LoraBank:
    """The adapters of one projection x [rows][K] -> [rows][N]; adapter i adds scales[i] (x a[i]^T) b[i]^T."""
    a: torch.Tensor                        # [adapters][slices][rank][K] (or [adapters][rank][K] with one slice)
    b: torch.Tensor                        # [adapters][N][rank]
    scales: torch.Tensor                   # float32 [adapters]
    ranks: Optional[torch.Tensor] = None   # int32 [adapters] (None: all of `rank`); what lies past a rank is not used
    slices: Optional[Tuple[int, ...]] = None  # columns of each slice (None: one slice of all N)

    def __post_init__(self):
        a, b = self.a, self.b
        _need(isinstance(a, torch.Tensor) and a.dim() in (3, 4), "a must be an [adapters][slices][rank][K] tensor")
        _need(isinstance(b, torch.Tensor) and b.dim() == 3, "b must be an [adapters][N][rank] tensor")
        n, r, K = a.shape[0], a.shape[-2], a.shape[-1]
        N = b.shape[1]
        S = a.shape[1] if a.dim() == 4 else 1
        slices = (N,) if self.slices is None else tuple(self.slices)
        _need(all(isinstance(w, int) and w > 0 for w in slices) and len(slices) == S and sum(slices) == N,
              lambda: f"slices must be {S} widths that add up to {N} columns, got {slices}")
        _dt(a.dtype)
        _check_tensor(a, "a", (a.dtype,), a.shape)
        _check_tensor(b, "b", (a.dtype,), (n, N, r), a.device)
        _check_tensor(self.scales, "scales", (torch.float32,), (n,), a.device)
        if self.ranks is not None:
            _check_tensor(self.ranks, "ranks", (torch.int32,), (n,), a.device)
        _need(n > 0, "a bank needs an adapter")
        ends, at = [], 0
        for w in slices:
            at += w
            ends.append(at)
        for name, v in (("count", n), ("rank", r), ("K", K), ("N", N), ("num_slices", S),
                        ("ends", (ctypes.c_int32 * S)(*ends))):
            object.__setattr__(self, name, v)


def wq_lora_workspace_bytes(rows: int, batch: int, K: int, rank: int, slices: int = 1) -> int:
    """Scratch of a wq_lora call with these sizes."""
    return int(lib().wq_lora_workspace_bytes(rows, batch, K, rank, slices))


def wq_lora(x: torch.Tensor, bank: LoraBank, adapters: torch.Tensor, y: torch.Tensor,
            cu_q: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, ws=None,
            stream=None) -> torch.Tensor:
    """y plus what each row's adapter makes of x: x [rows][K], y [rows][N], adapters int32 [batch] (the adapter of each
    sequence; a number that is not one of the bank's: none), cu_q as everywhere in the cache's functions (None: as many
    rows each).  out may be y itself.  ws: wq_lora_workspace_bytes() bytes of scratch, allocated when not given.  Rows
    outside every sequence of cu_q are left as they were in `out` (undefined where this call allocates it)."""
    if not (isinstance(x, torch.Tensor) and x.dim() == 2 and x.shape[1] == bank.K and x.is_contiguous()):
        raise ValueError("x must be a contiguous [rows][K] tensor")
    dtype, dev, rows = x.dtype, x.device, x.shape[0]
    dt = _dt(dtype)
    if bank.a.dtype != dtype or bank.a.device != dev:
        raise ValueError(f"the bank must be of x's dtype on its device, got {bank.a.dtype} on {bank.a.device}")
    shape = (rows, bank.N)
    for t, name in ((y, "y"), (out, "out")):
        if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.is_contiguous()
                and t.device == dev) and not (t is None and name == "out"):
            _check_tensor(t, name, (dtype,), shape, dev)
    if not (isinstance(adapters, torch.Tensor) and adapters.dim() == 1):
        raise ValueError("adapters must be a [batch] tensor")
    batch = adapters.shape[0]
    if not (adapters.dtype == torch.int32 and adapters.is_contiguous() and adapters.device == dev):
        _check_tensor(adapters, "adapters", (torch.int32,), (batch,), dev)
    if cu_q is not None:
        _check_tensor(cu_q, "cu_q", (torch.int32,), (batch + 1,), dev)
    elif rows and (batch == 0 or rows % batch):
        raise ValueError(f"without cu_q every sequence has as many rows: {rows} rows of {batch} sequences")
    if rows and batch == 0:
        raise ValueError("rows need a sequence")
    L = lib()
    need = L.wq_lora_workspace_bytes(rows, batch, bank.K, bank.rank, bank.num_slices)
    if ws is not None and need:
        _need(isinstance(ws, torch.Tensor) and ws.is_contiguous() and ws.device == dev,
              "ws must be a contiguous tensor on the device of x")
        _need(ws.numel() * ws.element_size() >= need, lambda: f"ws holds fewer than the {need} bytes this call needs")
    _check_cuda(x, "x")
    at = _stream(stream, dev)
    if out is None:
        out = _empty(stream, y, shape)
    if need and ws is None:
        ws = _empty(stream, x, need, torch.uint8, scratch=True)
    rc = L.wq_lora(x.data_ptr(), dt, bank.a.data_ptr(), bank.b.data_ptr(), bank.scales.data_ptr(), _ptr(bank.ranks),
                   adapters.data_ptr(), _ptr(cu_q), y.data_ptr(), out.data_ptr(), rows, batch, bank.count, bank.N,
                   bank.K, bank.rank, bank.num_slices, bank.ends, ws.data_ptr() if need else None, need, at)
    if rc:
        raise WQError("wq_lora", rc)
    return out
