"""References in 64 bits of the norm, rotary positions, adapters and page tables (CPU, no code of the package), each
with an elementwise bound on the error of the kernels' arithmetic."""
import math

import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # of the value, and of the smallest normal number
TINY = {torch.float16: 2.0 ** -14, torch.bfloat16: 2.0 ** -126}


def rounding(v, dt):
    """Half a step of `dt` at v (below the normal range: of its smallest normal number)."""
    return HALF_STEP[dt] * v.abs().clamp(min=TINY[dt])


def rms_norm(x, w, eps, residual=None):
    """(y, bound, h, bound).  The bound: the sum of squares has at most 64 + 6 + 16 additions one after another and the
    square's and h's own roundings, under 96 of 2^-24, halved by the root; 2^-21 for the root, the division and two
    products; the rounding to the type.  h is off by 2^-24 before its rounding."""
    dt = x.dtype
    h = x.double()
    if residual is not None:
        h = h + residual.double()
    size = torch.sqrt((h * h).sum(-1, keepdim=True) / h.shape[-1] + eps)
    y = w.double() * h / size
    rel = 48 * 2.0 ** -24 + 2.0 ** -21
    return y, y.abs() * rel * (1 + 2.0 ** -7) + rounding(y, dt), h, h.abs() * 2.0 ** -23 + rounding(h, dt)


def rotary(x, pos, freqs, axis, adjacent, factor):
    """x [T][H][D], pos [axes][T] -> (out, bound).  The bound: an angle in turns is p f / 2 pi to 2^-52 of it and cut
    at 2^-32; its remainder is held to 2^-24 of an eighth turn and sine and cosine add 2^-22; factor, two products and
    a sum 2^-22 of either channel; the rounding to the type."""
    T, H, D = x.shape
    half = len(freqs)
    f = torch.tensor(freqs, dtype=torch.float64)
    p = pos.double()[torch.tensor(axis)].t()       # [T][half]
    angle = p * f
    c, s = (angle.cos() * factor)[:, None], (angle.sin() * factor)[:, None]
    loose = ((p * f).abs() * 2.0 ** -52 + 2 * math.pi * 2.0 ** -32 + 2.0 ** -20)[:, None] * abs(factor)
    v, out = x.double(), x.double()
    i = torch.arange(half)
    one, two = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
    a, b = v[..., one], v[..., two]
    out[..., one], out[..., two] = a * c - b * s, a * s + b * c
    bound = torch.zeros_like(v)
    bound[..., one] = bound[..., two] = (a.abs() + b.abs()) * loose
    turned = torch.zeros(D, dtype=torch.bool)
    turned[:2 * half] = True
    return out, torch.where(turned, bound + rounding(out, x.dtype), torch.zeros_like(bound))


def lora(x, y, a, b, scales, ranks, slices, ids):
    """ids: the adapter of every row (below 0: none) -> (out, bound).  The bound: a sum over K has at most 32 additions
    inside a matrix instruction, K / 32 of them one after another and 64 over waves and parts; what it gives enters the
    second product in two parts, off by 2^-16 (bf16) or 2^-22 (fp16) of the row's largest; that one has at most
    2 rank + 8 additions; the scale, the sum with y (2^-22) and the rounding to the type."""
    dt, (T, K) = x.dtype, x.shape
    r = a.shape[-2]
    out, err = y.double(), torch.zeros(y.shape, dtype=torch.float64)
    u, parts = 2.0 ** -24, 2.0 ** -16 if dt == torch.bfloat16 else 2.0 ** -22
    ids_t = torch.tensor(ids)
    for i in sorted(set(ids)):
        if i < 0 or i >= a.shape[0]:
            continue
        rows = (ids_t == i).nonzero().flatten()
        X, k, at, w = x[rows].double(), ranks[i], 0, abs(float(scales[i]))
        for s, n in enumerate(slices):
            A, B = a[i, s, :k].double().t().contiguous(), b[i, at:at + n, :k].double().t().contiguous()
            v, mag = X @ A, X.abs() @ A.abs()
            ev = mag * (32 + K / 32 + 64) * u
            if k:
                ev = ev + parts * v.abs().amax(1, keepdim=True)
            delta = float(scales[i]) * (v @ B)
            out[rows, at:at + n] += delta
            err[rows, at:at + n] = (w * ((ev + (2 * r + 8) * u * v.abs()) @ B.abs()) * (1 + 2.0 ** -10)
                                    + (out[rows, at:at + n].abs() + delta.abs()) * 2.0 ** -22)
            at += n
    none = torch.tensor([not 0 <= i < a.shape[0] for i in ids])[:, None]
    return out, torch.where(none, torch.zeros_like(err), err + rounding(out, dt))


class Pages:
    """The page tables by their rules, one page at a time."""

    def __init__(self, table, lens, free, count, page):
        self.table, self.lens, self.free, self.count, self.page = [list(r) for r in table], list(lens), list(free), count, page
        self.lack = 0

    def resize(self, want, rows):
        P, width = self.page, len(self.table[0]) if self.table else 0
        pages = lambda n: -(-n // P)
        back = [(b, i) for b, (n, m) in enumerate(zip(self.lens, want)) for i in range(pages(max(m, 0)), pages(n))]
        take = [(b, i) for b, (n, m) in enumerate(zip(self.lens, want)) for i in range(pages(n), pages(m))]
        top = self.count + len(back)
        fails = any(m < 0 or m > width * P for m in want) or top > len(self.free)
        self.lack = -1 if fails else max(0, len(take) - top)
        if self.lack:
            return [0] * (len(want) + 1), [-1] * rows, [-1] * rows
        pool = [self.table[b][i] for b, i in back]
        for b, i in back:
            self.table[b][i] = -1
        for f in range(max(len(back), len(take))):
            page = pool[f] if f < len(back) else self.free[top - 1 - f]
            if f < len(take):
                self.table[take[f][0]][take[f][1]] = page
            else:
                self.free[top - 1 - f] = page
        self.count = top - len(take)
        cu, pos, slots = [0], [], []
        for b, (n, m) in enumerate(zip(self.lens, want)):
            pos += range(n, m)
            slots += [self.table[b][p // P] * P + p % P for p in range(n, m)]
            cu.append(len(pos))
        self.lens = list(want)
        fill = [-1] * max(0, rows - len(pos))
        return cu, (pos + fill)[:rows], (slots + fill)[:rows]
