"""Reference of the 4-bit key/value cache in 64 bits, from the definition in
include/wq.h (CPU, no code of the package), and helpers of its tests."""
import math

import torch

EPS = {torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}


def quantise(x, G):
    """x [T][H][D] (16-bit, CPU) -> codes, s, lo in float64, [T][H][D // G][G] / [T][H][D // G]."""
    dt = x.dtype
    g = x.double().reshape(x.shape[0], x.shape[1], x.shape[2] // G, G)
    bad = ~torch.isfinite(g).all(-1)
    g = torch.where(bad[..., None], torch.zeros_like(g), g)
    lo, hi = g.amin(-1), g.amax(-1)
    # half the range, so that it fits fp32: (max - min) / 15 rounded to fp32, then to the type
    half = (0.5 * hi - 0.5 * lo).float()
    s = (half.double() / 7.5).float().to(dt).double()
    t = (0.5 * g - 0.5 * lo[..., None]).float().double() * 2  # the 32-bit difference
    c = torch.where(s[..., None] > 0, torch.floor(t / s[..., None] + 0.5), torch.zeros_like(t)).clamp(0, 15)
    nan = torch.full_like(lo, math.nan)
    return c, torch.where(bad, torch.zeros_like(s), s), torch.where(bad, nan, lo)


def values(c, s, lo):
    """lo + s c in float64, [T][H][D]."""
    return (lo[..., None] + s[..., None] * c).flatten(2)


def stored(x, G):
    """What the cache gives back for the rows x, in their type: lo + s c (exact in 64 bits; s c alone may pass the
    range of fp32) held in fp32, rounded once."""
    return values(*quantise(x, G)).float().to(x.dtype)


def attention(q, K, V, pos, scale, causal, window, G, length=None):
    """One sequence.  q [n][Hq][D], K, V [L][H][D] (16-bit rows), pos [n] -> output and an
    elementwise bound on the error of the kernels' arithmetic, both float64 [n][Hq][D].

    The bound counts: the rounding of the output to its type (eps / 2); fp32 scores -- a dot product of
    D terms and the two terms of each group, each off by at most 2^-24 of sum |q| (|lo| + 15 s) per
    operation -- and the fp32 exponential (argument and result 2^-22 each), twice, since numerator and
    denominator carry them; p s rounded to fp16, 2^-11 of it, or half a subnormal step (2^-25 where the
    largest step stands at 4 or more) per key; the fp32 sums over the keys, 2^-24 per key."""
    n, Hq, D = q.shape
    H = K.shape[1]
    R, L = Hq // H, K.shape[0]
    kc, ks, klo = quantise(K, G)
    vc, vs, vlo = quantise(V, G)
    Kv, Vv = values(kc, ks, klo), values(vc, vs, vlo)
    Vmag = (vlo.abs()[..., None] + (vs[..., None] * vc)).flatten(2)
    Kmag = (klo.abs() + 15 * ks)[..., None].expand(-1, -1, -1, G).flatten(2)
    key = torch.arange(L)
    out = torch.zeros(n, Hq, D, dtype=torch.float64)
    bound = torch.zeros(n, Hq, D, dtype=torch.float64)
    seen = torch.ones(n, L, dtype=torch.bool)
    if causal:
        seen &= key[None] <= pos[:, None]
    if window:
        seen &= key[None] > pos[:, None] - window
    seen &= (pos >= 0)[:, None]
    alive = seen.any(1)
    for h in range(Hq if n and L else 0):
        kh = h // R
        qd = q[:, h].double()
        a = (qd @ Kv[:, kh].T) * scale
        mag = (qd.abs() @ Kmag[:, kh].nan_to_num(0).T) * scale
        a = torch.where(seen, a, torch.full_like(a, -math.inf))
        m = a.amax(1, keepdim=True)
        m = torch.where(alive[:, None], m, torch.zeros_like(m))
        p = torch.exp(a - m)
        p = torch.where(seen, p, torch.zeros_like(p))
        tot = p.sum(1, keepdim=True)
        w = p / torch.where(alive[:, None], tot, torch.ones_like(tot))
        # hidden keys may hold anything
        for i in range(n):
            if not alive[i]:
                continue
            ks_ = seen[i]
            wi = w[i, ks_]
            out[i, h] = wi @ Vv[ks_, kh]
            vm = wi @ Vmag[ks_, kh]
            amax = float(a[i, ks_].abs().max())
            ep = float(mag[i, ks_].max()) * (D + 8) * 2.0 ** -24 + 2.0 ** -22 * (2 + amax)
            smax = float(vs[ks_, kh].max())
            cnt = int(ks_.sum())
            bound[i, h] = vm * (2.0 ** -11 + 2 * ep + (cnt + 16) * 2.0 ** -24) + 15 * smax * 2.0 ** -27 * cnt
            bound[i, h] += EPS[q.dtype] / 2 * (out[i, h].abs() + bound[i, h]) + 2.0 ** -25
    return out, bound


class Problem:
    """Sequences over shuffled pages, with their histories, on the CPU; `fill` writes them with the library."""

    def __init__(self, lens, new, H, D, G, page, dt, seed, spare=3, scale=1.0, offset=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.new, self.H, self.D, self.G, self.page, self.dt = lens, new, H, D, G, page, dt
        used = [-(-n // page) for n in lens]
        self.num_pages = sum(used) + spare
        order = torch.randperm(self.num_pages, generator=g).tolist()
        self.table = torch.full((len(lens), max(max(used), 1) + 1), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.free = order[at:]
        shift = torch.randn(H, D, generator=g) * offset
        self.K = [((torch.randn(n, H, D, generator=g) + shift) * scale).to(dt) for n in lens]
        self.V = [(torch.randn(n, H, D, generator=g) * scale).to(dt) for n in lens]
        self.gen = g

    def cu(self, counts):
        out = [0]
        for c in counts:
            out.append(out[-1] + c)
        return torch.tensor(out, dtype=torch.int32)

    def empty(self, wq, device="cuda"):
        cache = wq.wq_kv_cache(self.num_pages, self.page, self.H, self.D, self.G, self.dt, device)
        cache.data.fill_(0xFF)  # NaN steps and offsets wherever nothing was written
        return cache

    def fill(self, wq, cache):
        k, v = torch.cat(self.K).cuda(), torch.cat(self.V).cuda()
        wq.wq_kv_write(k, v, cache, self.table.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(),
                       cu_q=self.cu(self.lens).cuda())

    def queries(self, Hq):
        return torch.randn(sum(self.new), Hq, self.D, generator=self.gen).to(self.dt)

    def reference(self, q, scale, causal=True, window=0):
        outs, bounds = [], []
        at = 0
        for b, n in enumerate(self.new):
            pos = torch.arange(self.lens[b] - n, self.lens[b])
            o, e = attention(q[at:at + n], self.K[b], self.V[b], pos, scale, causal, window, self.G)
            outs.append(o)
            bounds.append(e)
            at += n
        return torch.cat(outs), torch.cat(bounds)
