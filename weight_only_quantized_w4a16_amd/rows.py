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


def _rows(x, name: str, dtype, dim: Optional[int], dev, heads: Optional[int], rows: Optional[int]):
    """Address and elements between rows of x [rows][heads][dim] (a row contiguous)."""
    if not (isinstance(x, torch.Tensor) and x.dim() == 3):
        raise ValueError(f"{name} must be a [rows][heads][channels] tensor")
    n, h, d = x.shape
    sn, sh, sd = x.stride()
    if n <= 1:
        sn = h * d
    at = x.data_ptr()
    if ((dim is None or d == dim) and x.dtype == dtype and (rows is None or n == rows) and (heads is None or h == heads)
            and x.device == dev and (n == 0 or h == 0 or d == 0 or ((sd == 1 or d == 1) and (h == 1 or sh == d)
                                                                   and sn >= h * d and sn % 8 == 0 and at % 16 == 0))):
        return at, sn
    _need(x.dtype == dtype, f"{name} must have dtype {dtype}, got {x.dtype}")
    _need(dim is None or d == dim, f"{name} must have {dim} channels, got {d}")
    _need(heads is None or h == heads, f"{name} must have {heads} heads, got {h}")
    _need(rows is None or n == rows, f"{name} must have {rows} rows, got {n}")
    _need(x.device == dev, f"{name} must be on {dev}, got {x.device}")
    _need(sd == 1 and (h == 1 or sh == d), f"the heads of a row of {name} must be contiguous")
    _need(sn >= h * d and sn % 8 == 0, f"the row stride of {name} must be a multiple of 8 elements and hold a row")
    raise ValueError(f"{name} must be 16-byte aligned")


def wq_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                stream=None) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """y = weight h / sqrt(mean(h^2) + eps) over the last dimension, h = x (+ residual); with a residual the result is
    (y, h).  x [rows][channels], or [rows][heads][channels] (each head by itself).  out and sum_out (h's place) may be
    x or residual themselves."""
    if not (isinstance(x, torch.Tensor) and x.dim() in (2, 3)):
        raise ValueError("x must be a [rows][channels] or [rows][heads][channels] tensor")
    flat = x.dim() == 2

    def three(t, name):
        if not (isinstance(t, torch.Tensor) and t.dim() == x.dim()):
            raise ValueError(f"{name} must be a tensor like x")
        return t.unsqueeze(1) if flat else t

    dt, dev = _dt(x.dtype), x.device
    xs = three(x, "x")
    x_at, ld_x = _rows(xs, "x", x.dtype, None, dev, None, None)
    rows, heads, dim = xs.shape
    _need(heads > 0 and dim > 0, "x must have channels")
    _check_tensor(weight, "weight", (x.dtype,), (dim,), dev)
    r_at, ld_r = (None, 0) if residual is None else _rows(three(residual, "residual"), "residual", x.dtype, dim, dev,
                                                          heads, rows)
    if not (isinstance(eps, (int, float)) and eps > 0 and math.isfinite(eps)):
        raise ValueError(f"eps must be positive and finite, got {eps}")
    _need(sum_out is None or residual is not None, "sum_out needs a residual")
    if out is not None:
        y_at, ld_y = _rows(three(out, "out"), "out", x.dtype, dim, dev, heads, rows)
    if sum_out is not None:
        s_at, ld_s = _rows(three(sum_out, "sum_out"), "sum_out", x.dtype, dim, dev, heads, rows)
    _check_cuda(x, "x")
    at = _stream(stream, dev)
    if out is None:
        out = _empty(stream, x, x.shape)
        y_at, ld_y = out.data_ptr(), heads * dim
    if residual is None:
        s_at, ld_s = None, 0
    elif sum_out is None:
        sum_out = _empty(stream, x, x.shape)
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
    dt, dev, D = _dt(q.dtype), q.device, plan.head_dim
    q_at, ld_q = _rows(q, "q", q.dtype, D, dev, None, None)
    rows, heads = q.shape[0], q.shape[1]
    _need(heads > 0, "q must have heads")
    if k is None:
        k_at, ld_k, kv_heads = None, 0, 0
    else:
        k_at, ld_k = _rows(k, "k", q.dtype, D, dev, None, rows)
        kv_heads = k.shape[1]
        _need(kv_heads > 0, "k must have heads")
    if plan.turns.device != dev:
        raise ValueError("the plan and q must be on the same device")
    ld_pos = batch = 0
    if positions is not None:
        _need(kv_lens is None and cu_q is None, "either positions or kv_lens")
        shape = (rows,) if positions.dim() == 1 else (plan.num_axes, rows)
        _check_tensor(positions, "positions", (torch.int32,), shape, dev)
        ld_pos = rows if positions.dim() == 2 else 0
    else:
        _need(isinstance(kv_lens, torch.Tensor) and kv_lens.dim() == 1, "positions or kv_lens [batch] are needed")
        batch = kv_lens.shape[0]
        _check_tensor(kv_lens, "kv_lens", (torch.int32,), (batch,), dev)
        if cu_q is not None:
            _check_tensor(cu_q, "cu_q", (torch.int32,), (batch + 1,), dev)
        elif rows and (batch == 0 or rows % batch):
            raise ValueError(f"without cu_q every sequence has as many rows: {rows} rows of {batch} sequences")
        if rows and batch == 0:
            raise ValueError("rows need a sequence")
    if out is not None:
        q_out, k_out = out
        qo_at, ld_qo = _rows(q_out, "out[0]", q.dtype, D, dev, heads, rows)
        if k is None:
            _need(k_out is None, "out[1] must be None without k")
        else:
            ko_at, ld_ko = _rows(k_out, "out[1]", q.dtype, D, dev, kv_heads, rows)
    _check_cuda(q, "q")
    at = _stream(stream, dev)
    if out is None:
        q_out = _empty(stream, q, q.shape)
        qo_at, ld_qo = q_out.data_ptr(), heads * D
        k_out = None
        if k is not None:
            k_out = _empty(stream, k, k.shape)
            ko_at, ld_ko = k_out.data_ptr(), kv_heads * D
    if k is None:
        ko_at, ld_ko = None, 0
    rc = lib().wq_rotary(q_at, ld_q, k_at, ld_k, dt, plan.turns.data_ptr(), _ptr(plan.axis), plan.factor,
                         _ptr(positions), ld_pos, _ptr(kv_lens), _ptr(cu_q), qo_at, ld_qo, ko_at, ld_ko, rows, batch,
                         heads, kv_heads, D, plan.rotary_dim, int(plan.adjacent), plan.num_axes, at)
    if rc:
        raise WQError("wq_rotary", rc)
    return q_out, k_out
