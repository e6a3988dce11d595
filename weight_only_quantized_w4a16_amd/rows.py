"""Rows of a decoder layer between its products: root-mean-square norm with the residual's addition, and rotary
positions on queries and keys.

Like the rest of the package these functions only check and marshal arguments (arithmetic: include/wq.h).  Rows are
[rows][channels] or [rows][heads][channels], a row's heads contiguous, rows strided at will: slices of a fused
projection's output are taken as they are.  `stream` as in the cache's functions.
"""
from __future__ import annotations

import dataclasses
import math
from typing import Optional, Sequence, Tuple, Union

import torch

from . import WQError, _check_cuda, _check_tensor, _dt, _empty, _need, _ptr, _stream, lib


def _rows(x, name: str, dtype, shape, dev) -> Tuple[int, int]:
    """Address and elements between rows of x ([rows][channels] or [rows][heads][channels] of `shape`, a row contiguous)."""
    # (these checks run on every call: the common case first, what is wrong is named only after it failed)
    if isinstance(x, torch.Tensor) and x.shape == shape and x.dtype == dtype and x.device == dev:
        at, sn = x.data_ptr(), x.stride(0)
        if x.is_contiguous():
            if at % 16 == 0:
                return at, sn if shape[0] > 1 else shape[-1] * (shape[1] if len(shape) == 3 else 1)
        else:
            st = x.stride()
            width = shape[-1] * (shape[1] if len(shape) == 3 else 1)
            if not (st[-1] == 1 and (len(shape) == 2 or shape[1] == 1 or st[1] == shape[-1])):
                raise ValueError(f"a row of {name} (its heads, their channels) must be contiguous")
            if shape[0] > 1 and (sn < width or sn % 8):
                raise ValueError(f"the row stride of {name} must be a multiple of 8 elements and hold a row")
            if at % 16 == 0:
                return at, sn if shape[0] > 1 else width
        raise ValueError(f"{name} must be 16-byte aligned")
    _need(isinstance(x, torch.Tensor), f"{name} must be a tensor")
    _need(x.dtype == dtype, f"{name} must have dtype {dtype}, got {x.dtype}")
    _need(x.shape == shape, f"{name} must have shape {tuple(shape)}, got {tuple(x.shape)}")
    raise ValueError(f"{name} must be on {dev}, got {x.device}")


def wq_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                stream=None) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """y = weight h / sqrt(mean(h^2) + eps) over the last dimension, h = x (+ residual); with a residual the result is
    (y, h).  x [rows][channels], or [rows][heads][channels] (each head by itself).  out and sum_out (h's place) may be
    x or residual themselves."""
    if not (isinstance(x, torch.Tensor) and x.dim() in (2, 3)):
        raise ValueError("x must be a [rows][channels] or [rows][heads][channels] tensor")
    shape, dtype, dev = x.shape, x.dtype, x.device
    dt = _dt(dtype)
    rows, dim = shape[0], shape[-1]
    heads = shape[1] if len(shape) == 3 else 1
    if heads == 0 or dim == 0:
        raise ValueError("x must have channels")
    x_at, ld_x = _rows(x, "x", dtype, shape, dev)
    if not (isinstance(weight, torch.Tensor) and weight.dtype == dtype and weight.shape == (dim,) and weight.is_contiguous()
            and weight.device == dev):
        _check_tensor(weight, "weight", (dtype,), (dim,), dev)
    if not (isinstance(eps, (int, float)) and eps > 0 and math.isfinite(eps)):
        raise ValueError(f"eps must be positive and finite, got {eps}")
    r_at, ld_r, s_at, ld_s = None, 0, None, 0
    if residual is not None:
        r_at, ld_r = _rows(residual, "residual", dtype, shape, dev)
        if sum_out is not None:
            s_at, ld_s = _rows(sum_out, "sum_out", dtype, shape, dev)
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    if out is not None:
        y_at, ld_y = _rows(out, "out", dtype, shape, dev)
    _check_cuda(x, "x")
    at = _stream(stream, dev)
    plain = stream is None and x.is_contiguous()  # (a little cheaper than _empty)
    if out is None:
        out = torch.empty_like(x) if plain else _empty(stream, x, shape)
        y_at, ld_y = out.data_ptr(), heads * dim
    if residual is not None and sum_out is None:
        sum_out = torch.empty_like(x) if plain else _empty(stream, x, shape)
        s_at, ld_s = sum_out.data_ptr(), heads * dim
    rc = lib().wq_rms_norm(x_at, ld_x, r_at, ld_r, weight.data_ptr(), eps, dt, y_at, ld_y, s_at, ld_s, rows, heads,
                           dim, at)
    if rc:
        raise WQError("wq_rms_norm", rc)
    return out if residual is None else (out, sum_out)


@dataclasses.dataclass(frozen=True)
class Rotary:
    """What rotary positions need besides the rows (made by wq_rotary_plan)."""
    turns: torch.Tensor             # int64 [rotary_dim / 2]: the turn per position, in units of 2^-64
    axis: Optional[torch.Tensor]    # int32 [rotary_dim / 2]: each pair's axis (None: one axis)
    num_axes: int
    head_dim: int
    rotary_dim: int
    adjacent: bool
    factor: float

    def __post_init__(self):
        for name in ("num_axes", "head_dim", "rotary_dim"):
            v = getattr(self, name)
            _need(isinstance(v, int) and 0 < v < 1 << 16, f"{name} must be a positive count, got {v!r}")
        _need(self.rotary_dim % 2 == 0 and self.rotary_dim <= self.head_dim,
              "rotary_dim must be even and at most head_dim")
        _check_tensor(self.turns, "turns", (torch.int64,), (self.rotary_dim // 2,))
        if self.axis is not None:
            _check_tensor(self.axis, "axis", (torch.int32,), (self.rotary_dim // 2,), self.turns.device)
        _need(self.axis is not None or self.num_axes == 1, "several axes need each pair's axis")
        _need(math.isfinite(self.factor), "factor must be finite")


def wq_rotary_plan(head_dim: int, rotary_dim: Optional[int] = None, base: float = 10000.0,
                   freqs: Optional[Sequence[float]] = None, sections: Optional[Sequence[int]] = None,
                   axes: Optional[Sequence[int]] = None, adjacent: bool = False, factor: float = 1.0,
                   device="cuda") -> Rotary:
    """Rotary positions of head_dim channels, the first rotary_dim of them turning (default: all).

    freqs: angle per position of each of the rotary_dim / 2 pairs, in radians (default base ** (-2 i / rotary_dim);
    scaled ones of long-context models go here).  sections: several axes, how many consecutive pairs each has; or axes:
    the axis of every pair.  adjacent: pairs are neighbouring channels (default: channels rotary_dim / 2 apart).
    factor multiplies the turned channels."""
    rotary_dim = head_dim if rotary_dim is None else rotary_dim
    half = rotary_dim // 2
    if freqs is None:
        _need(base > 0 and math.isfinite(base), lambda: f"base must be positive and finite, got {base}")
        freqs = [base ** (-2.0 * i / rotary_dim) for i in range(half)]
    else:
        freqs = torch.as_tensor(freqs, dtype=torch.float64).tolist()
    _need(len(freqs) == half, lambda: f"{half} pairs need as many frequencies, got {len(freqs)}")
    _need(all(math.isfinite(f) for f in freqs), "frequencies must be finite")
    _need(sections is None or axes is None, "either sections or axes")
    if sections is not None:
        _need(all(isinstance(n, int) and n >= 0 for n in sections) and sum(sections) == half,
              lambda: f"sections must add up to the {half} pairs, got {list(sections)}")
        axes = [a for a, n in enumerate(sections) for _ in range(n)]
        num = max(1, len(sections))
    elif axes is not None:
        axes = [int(a) for a in axes]
        _need(len(axes) == half and min(axes) >= 0, lambda: f"axes must name one axis for each of the {half} pairs")
        num = max(axes) + 1
    else:
        num = 1
    u = []
    for f in freqs:
        t = f / (2 * math.pi)
        v = int((t - math.floor(t)) * 2.0 ** 64) % (1 << 64)
        u.append(v - (1 << 64) if v >= 1 << 63 else v)
    return Rotary(torch.tensor(u, dtype=torch.int64, device=device),
                  torch.tensor(axes, dtype=torch.int32, device=device) if num > 1 else None, num, head_dim, rotary_dim,
                  bool(adjacent), float(factor))


def wq_rotary(q: torch.Tensor, k: Optional[torch.Tensor], plan: Rotary, positions: Optional[torch.Tensor] = None,
              kv_lens: Optional[torch.Tensor] = None, cu_q: Optional[torch.Tensor] = None, out=None,
              stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Queries q and keys k ([rows][heads][head_dim]; k may be None) turned to their positions.

    positions int32 [rows] (all axes alike) or [axes][rows]; or kv_lens (and cu_q), as everywhere in the cache's
    functions: a sequence's rows are its last ones.  out: the pair the results go to, which may be (q, k) itself.  Rows
    outside every sequence of cu_q are left as they were in `out` (undefined where this call allocates it)."""
    if not (isinstance(q, torch.Tensor) and q.dim() == 3):
        raise ValueError("q must be a [rows][heads][head_dim] tensor")
    shape, dtype, dev, D = q.shape, q.dtype, q.device, plan.head_dim
    dt = _dt(dtype)
    rows, heads, d = shape
    if d != D or heads == 0:
        raise ValueError(f"q must have heads of {D} channels, got {tuple(shape)}")
    q_at, ld_q = _rows(q, "q", dtype, shape, dev)
    k_at, ld_k, kv_heads, ko_at, ld_ko = None, 0, 0, None, 0
    if k is not None:
        k_shape = k.shape if isinstance(k, torch.Tensor) else ()
        if len(k_shape) != 3 or k_shape[0] != rows or k_shape[1] == 0 or k_shape[2] != D:
            raise ValueError(f"k must be [{rows}][heads][{D}], got {tuple(k_shape)}")
        k_at, ld_k = _rows(k, "k", dtype, k_shape, dev)
        kv_heads = k_shape[1]
    if plan.turns.device != dev:
        raise ValueError("the plan and q must be on the same device")
    ld_pos = batch = 0
    if positions is not None:
        _need(kv_lens is None and cu_q is None, "either positions or kv_lens")
        _need(isinstance(positions, torch.Tensor), "positions must be a tensor")
        _check_tensor(positions, "positions", (torch.int32,), (rows,) if positions.dim() == 1 else (plan.num_axes, rows),
                      dev)
        ld_pos = rows if positions.dim() == 2 else 0
    else:
        _need(isinstance(kv_lens, torch.Tensor) and kv_lens.dim() == 1, "positions or kv_lens [batch] are needed")
        batch = kv_lens.shape[0]
        if not (kv_lens.dtype == torch.int32 and kv_lens.is_contiguous() and kv_lens.device == dev):
            _check_tensor(kv_lens, "kv_lens", (torch.int32,), (batch,), dev)
        if cu_q is not None:
            _check_tensor(cu_q, "cu_q", (torch.int32,), (batch + 1,), dev)
        elif rows and (batch == 0 or rows % batch):
            raise ValueError(f"without cu_q every sequence has as many rows: {rows} rows of {batch} sequences")
        if rows and batch == 0:
            raise ValueError("rows need a sequence")
    if out is not None:
        q_out, k_out = out
        qo_at, ld_qo = _rows(q_out, "out[0]", dtype, shape, dev)
        if k is not None:
            ko_at, ld_ko = _rows(k_out, "out[1]", dtype, k_shape, dev)
        elif k_out is not None:
            raise ValueError("out[1] must be None without k")
    _check_cuda(q, "q")
    at = _stream(stream, dev)
    if out is None:
        q_out, k_out = _empty(stream, q, shape), None
        qo_at, ld_qo = q_out.data_ptr(), heads * D
        if k is not None:
            k_out = _empty(stream, k, k_shape)
            ko_at, ld_ko = k_out.data_ptr(), kv_heads * D
    rc = lib().wq_rotary(q_at, ld_q, k_at, ld_k, dt, plan.turns.data_ptr(), _ptr(plan.axis), plan.factor,
                         _ptr(positions), ld_pos, _ptr(kv_lens), _ptr(cu_q), qo_at, ld_qo, ko_at, ld_ko, rows, batch,
                         heads, kv_heads, D, plan.rotary_dim, int(plan.adjacent), plan.num_axes, at)
    if rc:
        raise WQError("wq_rotary", rc)
    return q_out, k_out
