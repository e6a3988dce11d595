"""Attention over the 4-bit cache where steps of one call differ by many powers of two -- values of keys a row does not
see, of keys that count for nothing, of keys that count alike; key groups far below the others -- and where memory that
no row sees holds anything."""
import math

import pytest
import torch

import _kv

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def wq():
    import weight_only_quantized_w4a16_amd as m
    m.lib()
    assert torch.cuda.is_available()
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def reference(q, K, V, pos, scale, G, causal=True, window=0):
    """_kv.attention's output with a bound that follows the steps a row sees, [n][Hq][D] in 64 bits.

    Per key of probability w (64-bit, summing to 1), step s, value v = lo + s c:
      * w s rounded to fp16 and the score's errors, w |v| (2^-11 + 2 ep + 2^-24 per key), as in _kv.attention;
      * where w s is small against the row's largest, the fp16 number is a subnormal: the row's reference puts its
        largest w s at 2^6 or more, half a subnormal step is 2^-25, and 2^4 times that for the keys whose code
        carries a factor of 2^4: 2^-21 / 2^6 of the largest w s, times v / s (|lo| / s + c, 1 in a group without a
        step);
      * lo / s held in two fp16, half a subnormal step 2^-25 of the second, times 2^4 where it is stored times 2^-4:
        2^-21 w s;
    then the output's own rounding."""
    n, Hq, D = q.shape
    H = K.shape[1]
    out, _ = _kv.attention(q, K, V, pos, scale, causal, window, G)
    kc, ks, klo = _kv.quantise(K, G)
    vc, vs, vlo = _kv.quantise(V, G)
    Kv = _kv.values(kc, ks, klo)
    Kmag = (klo.abs() + 15 * ks)[..., None].expand(-1, -1, -1, G).flatten(2)
    Vmag = (vlo.abs()[..., None] + vs[..., None] * vc).flatten(2)
    flat = (vs == 0)[..., None]
    step = torch.where(vs > 0, vs, vlo.abs())
    ratio = vlo.abs()[..., None] / vs.clamp_min(1e-300)[..., None]
    times = torch.where(flat, torch.ones_like(vc), ratio + vc).flatten(2)
    steps = step[..., None].expand(-1, -1, -1, G).flatten(2)
    key = torch.arange(K.shape[0])
    bound = torch.zeros_like(out)
    for i in range(n):
        seen = torch.full_like(key, int(pos[i]) >= 0, dtype=torch.bool)
        if causal:
            seen &= key <= pos[i]
        if window:
            seen &= key > pos[i] - window
        if not bool(seen.any()):
            continue
        for h in range(Hq):
            kh = h // (Hq // H)
            a = Kv[seen, kh] @ q[i, h].double() * scale
            mag = float((Kmag[seen, kh] @ q[i, h].double().abs()).max()) * scale
            w = torch.softmax(a, 0)
            ep = mag * (D + 8) * 2.0 ** -24 + 2.0 ** -22 * (2 + float(a.abs().max()))
            largest = float((w * step[seen, kh].amax(1)).max())
            b = (w @ Vmag[seen, kh]) * (2.0 ** -11 + 2 * ep + (int(seen.sum()) + 16) * 2.0 ** -24)
            b += 2.0 ** -27 * largest * times[seen, kh].sum(0) + 2.0 ** -21 * (w @ steps[seen, kh])
            half = _kv.EPS[q.dtype] / 2
            bound[i, h] = b + half * (out[i, h].abs() + b) + half * torch.finfo(q.dtype).tiny
    return out, bound


def run(wq, P, q, **kw):
    cache = P.empty(wq)
    P.fill(wq, cache)
    return wq.wq_kv_attention(q.cuda(), cache, P.table.cuda(), i32(P.lens), **kw).cpu().double()


def worst(err, bound):
    """Largest error in bounds (NaN counts as infinite)."""
    return float(torch.where(err.isnan(), torch.full_like(err, math.inf), err / bound).max())


# ---------------------------------------------------------------------------
# Keys a row does not see
# ---------------------------------------------------------------------------
HIDDEN = [(F16, 2.0 ** -9, 2.0 ** 18), (F16, 2.0 ** -9, 2.0 ** 21), (BF16, 1.0, 2.0 ** 24), (BF16, 1.0, 2.0 ** 40),
          (BF16, 2.0 ** -50, 2.0 ** 120)]


@pytest.mark.parametrize("dt,base,factor", HIDDEN)
@pytest.mark.parametrize("D,G,heads,new", [(64, 64, 2, 64), (64, 64, 1, 12), (128, 64, 4, 40), (128, 128, 4, 5),
                                           (256, 64, 2, 30)])
def test_larger_values_of_later_tokens(wq, dt, base, factor, D, G, heads, new):
    """The last tokens of a prompt hold far larger values: the rows before them do not change."""
    P = _kv.Problem([64 + 5], [new], 1, D, G, 16, dt, D + new, scale=1.0)
    P.V[0] = P.V[0] * base
    q = P.queries(heads)
    pos = torch.arange(69 - new, 69)
    P.V[0][-2:] = (P.V[0][-2:].double() * factor).to(dt)
    assert bool(P.V[0].isfinite().all())
    got = run(wq, P, q)
    want, bound = reference(q, P.K[0], P.V[0], pos, D ** -0.5, G)
    err = (got - want).abs() / base
    assert worst(err[:-2], bound[:-2] / base) <= 1, worst(err[:-2], bound[:-2] / base)
    assert worst(err[-2:], bound[-2:] / base) <= 1  # the rows that see them


@pytest.mark.parametrize("dt,base,factor", HIDDEN)
@pytest.mark.parametrize("new", [1, 3, 40])
def test_larger_values_before_the_window(wq, dt, base, factor, new):
    """Positions just before the window, in the window's first block of 64, hold far larger values."""
    n, window = 200, 50
    P = _kv.Problem([n], [new], 1, 64, 32, 16, dt, new)
    P.V[0] = P.V[0] * base
    first = n - new - window + 1  # the first row's window begins here
    P.V[0][first - 2:first] = (P.V[0][first - 2:first].double() * factor).to(dt)
    q = P.queries(2)
    got = run(wq, P, q, window=window)
    want, bound = reference(q, P.K[0], P.V[0], torch.arange(n - new, n), 0.125, 32, window=window)
    assert worst((got - want).abs(), bound) <= 1
    if new > 1:  # seen by the first rows, hidden from the rest
        P.V[0][first - 2:first] = P.V[0][first - 4:first - 2]
        P.V[0][first] = (P.V[0][first].double() * factor).to(dt)
        got = run(wq, P, q, window=window)
        want, bound = reference(q, P.K[0], P.V[0], torch.arange(n - new, n), 0.125, 32, window=window)
        assert worst((got - want).abs(), bound) <= 1


@pytest.mark.parametrize("dt,base,factor", HIDDEN[:4])
def test_larger_values_of_no_account(wq, dt, base, factor):
    """A key with far larger values that every row sees with next to no probability."""
    P = _kv.Problem([300], [20], 1, 64, 64, 16, dt, 5)
    P.V[0] = P.V[0] * base
    q = P.queries(2)
    q[:, :, 0] = 8.0
    P.K[0][:, :, 0] = 0
    P.K[0][100, :, 0] = -math.log2(factor)  # a probability of about factor^-1.44
    P.V[0][100] = (P.V[0][100].double() * factor).to(dt)
    got = run(wq, P, q)
    want, bound = reference(q, P.K[0], P.V[0], torch.arange(280, 300), 0.125, 64)
    assert worst((got - want).abs(), bound) <= 1


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("sink", [1.0, 2.0 ** -12, 0.0])
@pytest.mark.parametrize("new", [1, 40])
def test_a_sink_and_a_long_tail(wq, dt, sink, new):
    """One key takes nearly all of the probability; thousands of others, alike, share the rest."""
    n = 9000
    P = _kv.Problem([n], [new], 1, 64, 64, 64, dt, 6)
    q = P.queries(1)
    q[:, :, 0] = 8.0
    P.K[0] *= 0.01
    P.K[0][0, :, 0] = 15.0  # e^-15 (2^-21.6) for each of the others
    P.V[0] = P.V[0] + 1
    P.V[0][0] *= sink
    got = run(wq, P, q)
    want, bound = reference(q, P.K[0], P.V[0], torch.arange(n - new, n), 0.125, 64)
    assert worst((got - want).abs(), bound) <= 1


@pytest.mark.parametrize("lens,new", [([5000], [1]), ([5000], [20]), ([700], [1])])
def test_sums_over_steps_far_apart(wq, lens, new):
    """Half of the keys, all of the first ones, hold zeros; the others hold large values: their probabilities count
    alike, also where parts and waves are joined."""
    P = _kv.Problem(lens, new, 1, 64, 64, 16, BF16, 7)
    n = lens[0]
    P.V[0] = ((P.V[0].double() + 3) * 2.0 ** 90).to(BF16)
    P.V[0][:n // 2] = 0
    q = P.queries(2)
    got = run(wq, P, q)
    want, bound = reference(q, P.K[0], P.V[0], torch.arange(n - new[0], n), 0.125, 64)
    assert worst((got - want).abs() * 2.0 ** -90, bound * 2.0 ** -90) <= 1


@pytest.mark.parametrize("dt", [F16, BF16])
def test_scores_far_below_zero(wq, dt):
    """Rows whose scores are all far below zero still have a softmax."""
    top = 2.0 ** 10
    P = _kv.Problem([150], [40], 1, 64, 64, 16, dt, 8)
    q = P.queries(2) * 0
    q[:, :, 0] = -top
    P.K[0] *= 0
    P.K[0][:, :, 0] = top
    P.K[0][::7, :, 0] = top * 1.5  # these are left with nothing
    got = run(wq, P, q)
    keep = torch.arange(150) % 7 != 0
    v = _kv.values(*_kv.quantise(P.V[0], 64))[:, 0]
    for i in range(40):
        seen = keep & (torch.arange(150) <= 110 + i)
        want = v[seen].mean(0)
        # equal probabilities 1 / n: p s rounded to fp16, the output to its type, fp32 sums
        bound = v[seen].abs().mean(0) * 2.0 ** -11 + 8 * 2.0 ** -11 + _kv.EPS[dt] / 2 * (want.abs() + 0.01) + 2.0 ** -15
        assert bool(((got[i] - want).abs() <= bound).all()), i


# ---------------------------------------------------------------------------
# Memory nothing was written to
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_unwritten_pages_before_the_window(wq, dt, new):
    """Pages wholly before the window may name a page that was never written: infinite steps and offsets, offsets far
    larger than their steps, NaN, anything."""
    inf = 0x7C00 if dt == F16 else 0x7F80
    big = 0x7BFF if dt == F16 else 0x7F7F
    n, window = 230, 75
    first = n - new - window + 1
    pages = first // 16  # pages before the one the window begins in
    assert pages % 4  # the block of 64 keys holds a page before the window
    P = _kv.Problem([n], [new], 1, 64, 64, 16, dt, 60 + new)
    q = P.queries(2)
    want, bound = reference(q, P.K[0], P.V[0], torch.arange(n - new, n), 0.125, 64, window=window)
    for s, lo in ((inf, inf), (inf, 0), (1, big), (1, big | 0x8000), (0x3C00, inf), (0x8001, inf | 0x8000),
                  (0xFFFF, 0xFFFF)):
        cache = P.empty(wq)
        P.fill(wq, cache)
        word = (s | lo << 16)
        word -= (word >> 31) << 32
        spare = P.free[0]
        per = cache.data.numel() // P.num_pages
        cache.data[spare * per:(spare + 1) * per].view(torch.int32).fill_(word)
        table = P.table.clone()
        table[0, :pages] = spare
        got = wq.wq_kv_attention(q.cuda(), cache, table.cuda(), i32([n]), scale=0.125, window=window).cpu().double()
        assert worst((got - want).abs(), bound) <= 1, (hex(s), hex(lo))


# ---------------------------------------------------------------------------
# Key steps
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("e", [-40, -90, -101, -110, -120, -128])
@pytest.mark.parametrize("D,G,new", [(64, 64, 1), (64, 32, 1), (64, 32, 40), (128, 128, 40), (128, 64, 3)])
def test_tiny_key_groups(wq, e, D, G, new):
    """A group of keys far below the others adds next to nothing to a score, down to the subnormals of the type."""
    P = _kv.Problem([150], [new], 1, D, G, 16, BF16, e + 200 + D)
    P.K[0][:, :, :G] = (P.K[0][:, :, :G].double() * 2.0 ** e).to(BF16)
    q = P.queries(2)
    got = run(wq, P, q)
    want, bound = reference(q, P.K[0], P.V[0], torch.arange(150 - new, 150), D ** -0.5, G)
    assert worst((got - want).abs(), bound) <= 1


@pytest.mark.parametrize("e", [90, 97, 104])
@pytest.mark.parametrize("new", [1, 40])
def test_tiny_keys_meet_large_queries(wq, e, new):
    """Keys around 2^-e and queries around 2^e: ordinary scores."""
    P = _kv.Problem([150], [new], 1, 64, 64, 16, BF16, e)
    P.K[0] = (P.K[0].double() * 2.0 ** -e).to(BF16)
    q = (P.queries(2).double() * 2.0 ** e).to(BF16)
    got = run(wq, P, q)
    want, bound = reference(q, P.K[0], P.V[0], torch.arange(150 - new, 150), 0.125, 64)
    assert worst((got - want).abs(), bound) <= 1


# ---------------------------------------------------------------------------
# Scores
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("scale", [2.0 ** -6, 0.25, 1.0])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_beyond_the_fraction_of_fp32(wq, new, scale, sign):
    """Scores of 2^24 scale, where fp32 holds whole numbers at best: a later block's scores lie above the first one's
    by anything between nothing and all, and the output stays between the two blocks' values, at the second's where
    that has the weight whichever way the scores are rounded (each by up to 2^-22 of itself: the dot product's sums
    and the product with scale log2 e)."""
    n = 128 + 40
    off = 2.0 ** -22 * 2.0 ** 24 * scale * 2
    for step in [0.0] + [2.0 ** e * m for e in range(0, 6) for m in (1.0, 1.5)]:
        P = _kv.Problem([n], [new], 1, 64, 32, 16, F16, 1)
        P.K[0] = torch.zeros(n, 1, 64, dtype=F16)
        P.K[0][:, :, :32] = 8192.0 * sign      # groups of equal channels: held exactly
        P.K[0][64:, :, 32:] = step / scale
        P.V[0] = torch.linspace(1, 2, 64).half().repeat(n, 1, 1)
        P.V[0][64:] += 4
        q = torch.zeros(new, 2, 64, dtype=F16)
        q[:, :, 0], q[:, :, 32] = 2048.0, 1.0
        got = run(wq, P, q, scale=scale)
        a, b = (_kv.stored(P.V[0], 32)[i, 0].double() for i in (0, 64))
        tol = 8 * 2.0 ** -10
        assert bool(got.isfinite().all()), step
        assert bool(((got >= a - tol) & (got <= b + tol)).all()), step
        if step - off > 12:
            assert bool(((got - b).abs() <= tol + 4 * 64 * math.exp(-12)).all()), step
