"""The 4-bit key/value cache on the GPU against the 64-bit reference of
tests/_kv.py: rows written and read back bit for bit, attention within the
bound that counts its roundings."""
import math

import pytest
import torch

import _kv

pytestmark = pytest.mark.gpu

SHAPES = [(64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (192, 32), (192, 64), (256, 32), (256, 64),
          (256, 128)]
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def wq():
    import weight_only_quantized_w4a16_amd as m
    m.lib()
    assert torch.cuda.is_available()
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def same_bits(a, b):
    """Equal bit patterns; a NaN equals any NaN."""
    a, b = a.cpu(), b.cpu()
    return bool(((a.view(torch.int16) == b.view(torch.int16)) | (a.isnan() & b.isnan())).all())


def read_all(wq, P, cache):
    k, v = wq.wq_kv_read(cache, P.table.cuda(), i32(P.lens), sum(P.lens), cu_q=P.cu(P.lens).cuda())
    return k.cpu(), v.cpu()


# ---------------------------------------------------------------------------
# Rows in and out
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("D,G", SHAPES)
def test_write_read_every_shape(wq, D, G, dt):
    P = _kv.Problem([1, 37, 16, 70], None, 3, D, G, 16 if D != 128 else 32, dt, D + G)
    cache = P.empty(wq)
    P.fill(wq, cache)
    k, v = read_all(wq, P, cache)
    assert same_bits(k, _kv.stored(torch.cat(P.K), G))
    assert same_bits(v, _kv.stored(torch.cat(P.V), G))


@pytest.mark.parametrize("page", [16, 64, 1024])
def test_append_in_pieces(wq, page):
    """The same rows written in any pieces give the same cache, and a piece leaves every other row alone."""
    P = _kv.Problem([67, 130], None, 2, 128, 64, page, F16, 5)
    cache = P.empty(wq)
    table = P.table.cuda()
    pieces = [(0, 0), (1, 5), (14, 18), (16, 19), (17, 50), (31, 100), (64, 129), (66, 129), (67, 130)]
    at = (0, 0)
    for to in pieces:
        counts = [to[b] - at[b] for b in range(2)]
        k = torch.cat([P.K[b][at[b]:to[b]] for b in range(2)]).cuda()
        v = torch.cat([P.V[b][at[b]:to[b]] for b in range(2)]).cuda()
        wq.wq_kv_write(k, v, cache, table, i32(list(to)), cu_q=P.cu(counts).cuda())
        at = to
    k, v = read_all(wq, P, cache)
    assert same_bits(k, _kv.stored(torch.cat(P.K), 64)) and same_bits(v, _kv.stored(torch.cat(P.V), 64))
    # rewriting rows 20..22 of the first sequence (length cut back to 23) changes nothing else
    new_k, new_v = -P.K[0][20:23], P.V[0][20:23] * 2
    wq.wq_kv_write(new_k.cuda(), new_v.cuda(), cache, table[:1], i32([23]))
    P.K[0][20:23], P.V[0][20:23] = new_k, new_v
    k, v = read_all(wq, P, cache)
    assert same_bits(k, _kv.stored(torch.cat(P.K), 64)) and same_bits(v, _kv.stored(torch.cat(P.V), 64))


@pytest.mark.parametrize("batch", [1, 3, 64, 65, 300])
def test_single_tokens_of_many_sequences(wq, batch):
    """Decode step: one row each, with and without row offsets, some sequences without a row."""
    lens = [1 + (7 * b) % 41 for b in range(batch)]
    P = _kv.Problem(lens, None, 2, 64, 64, 16, BF16, batch)
    cache = P.empty(wq)
    last_k, last_v = torch.stack([k[-1] for k in P.K]), torch.stack([v[-1] for v in P.V])
    wq.wq_kv_write(last_k.cuda(), last_v.cuda(), cache, P.table.cuda(), i32(lens))
    k, v = wq.wq_kv_read(cache, P.table.cuda(), i32(lens), batch)
    assert same_bits(k, _kv.stored(last_k, 64)) and same_bits(v, _kv.stored(last_v, 64))
    cache = P.empty(wq)
    counts = [b % 3 for b in range(batch)]
    counts = [min(c, n) for c, n in zip(counts, lens)]
    rows = sum(counts)
    cu = P.cu(counts).cuda()
    kk = torch.cat([P.K[b][lens[b] - c:] for b, c in enumerate(counts)])
    vv = torch.cat([P.V[b][lens[b] - c:] for b, c in enumerate(counts)])
    wq.wq_kv_write(kk.cuda(), vv.cuda(), cache, P.table.cuda(), i32(lens), cu_q=cu)
    k, v = wq.wq_kv_read(cache, P.table.cuda(), i32(lens), rows, cu_q=cu)
    assert same_bits(k, _kv.stored(kk, 64)) and same_bits(v, _kv.stored(vv, 64))


@pytest.mark.parametrize("dt", [F16, BF16])
def test_values_at_the_borders(wq, dt):
    """Half-way values (a symmetric range puts 0 between two codes), constant groups, subnormals, the largest
    values of the type, infinities and NaN."""
    D = G = 64
    rows = torch.zeros(16, 1, D, dtype=torch.float64)
    base = torch.linspace(-1, 1, D, dtype=torch.float64)
    tiny = float(torch.finfo(dt).tiny) * float(torch.finfo(dt).eps)  # the smallest subnormal
    big = float(torch.finfo(dt).max)
    rows[0, 0] = base
    rows[1, 0] = torch.where(torch.arange(D) % 3 == 0, base, torch.zeros(D, dtype=torch.float64))
    rows[2, 0] = 3.25
    rows[3, 0] = 0.0
    rows[4, 0] = torch.arange(D) % 16 * tiny
    rows[5, 0] = torch.arange(D) % 5 * tiny
    rows[6, 0] = (torch.arange(D) % 31 - 15) * 0.5     # steps of 1, every half in the range
    rows[7, 0] = base * big
    rows[8, 0] = torch.where(torch.arange(D) < 3, torch.full((D,), -big, dtype=torch.float64), base * 1e-3)
    rows[9, 0] = 1000 + base
    rows[10, 0] = base
    rows[11, 0] = base
    rows[12, 0] = (torch.arange(D) - 7.5) * 2.0 ** -20 * (1 if dt == F16 else 2.0 ** -100)
    rows[13, 0] = torch.where(torch.arange(D) == 5, torch.full((D,), tiny, dtype=torch.float64), -rows[1, 0])
    x = rows.to(dt)
    x[10, 0, 17] = math.inf
    x[11, 0, 3] = math.nan
    P = _kv.Problem([16], None, 1, D, G, 16, dt, 1)
    P.K, P.V = [x], [x]
    cache = P.empty(wq)
    P.fill(wq, cache)
    k, v = read_all(wq, P, cache)
    want = _kv.stored(x, G)
    for i in range(16):
        assert same_bits(k[i], want[i]), i
        assert same_bits(v[i], want[i]), i
    assert bool(k[10:12].isnan().all()) and not bool(k[9].isnan().any())


def test_strided_rows(wq):
    """Keys and values as slices of a fused projection's output, read back into another wide buffer."""
    T, H, D = 41, 2, 128
    qkv = torch.randn(T, (4 + 2 * H) * D).half().cuda()
    k = qkv[:, 4 * D:(4 + H) * D].view(T, H, D)
    v = qkv[:, (4 + H) * D:].view(T, H, D)
    cache = wq.wq_kv_cache(5, 16, H, D, 128, F16)
    table = i32([[4, 0, 2]])
    wq.wq_kv_write(k, v, cache, table, i32([T]))
    wide = torch.full((T, 3 * H * D), 7.0, dtype=F16, device="cuda")
    out = (wide[:, :H * D].view(T, H, D), wide[:, 2 * H * D:].view(T, H, D))
    wq.wq_kv_read(cache, table, i32([T]), T, out=out)
    assert same_bits(out[0].contiguous(), _kv.stored(k.cpu().contiguous(), 128))
    assert same_bits(out[1].contiguous(), _kv.stored(v.cpu().contiguous(), 128))
    assert bool((wide[:, H * D:2 * H * D] == 7).all())


def test_rows_without_a_place(wq):
    """Missing pages, lengths below the rows, lengths past the table and rows outside every sequence: nothing else
    is written, such rows read as zero, rows of no sequence stay as they were."""
    H, D, G = 1, 64, 64
    cache = wq.wq_kv_cache(4, 16, H, D, G, F16)
    cache.data.fill_(0x11)
    before = cache.data.clone()
    table = i32([[0, -1, 1], [7, 2, -1], [4, -5, 2 ** 31 - 1]])
    lens = i32([40, 3, 999])
    cu = i32([2, 42, 47, 60])  # rows 0, 1 and 60.. belong to nobody; sequence 1 has 5 rows for 3 positions
    x = torch.randn(64, H, D).half().cuda()
    wq.wq_kv_write(x, x, cache, table, lens, cu_q=cu)
    rec = before.numel() // 4
    changed = [not torch.equal(cache.data[p * rec:(p + 1) * rec], before[p * rec:(p + 1) * rec]) for p in range(4)]
    assert changed == [True, True, False, False]
    k = torch.full((64, H, D), 5.0, dtype=F16, device="cuda")
    v = k.clone()
    wq.wq_kv_read(cache, table, lens, 64, cu_q=cu, out=(k, v))
    want = _kv.stored(x.cpu(), G)
    for got in (k.cpu(), v.cpu()):
        assert bool((got[:2] == 5).all()) and bool((got[60:] == 5).all())
        assert same_bits(got[2:18], want[2:18]) and same_bits(got[34:42], want[34:42])
        assert bool((got[18:34] == 0).all())   # page -1
        assert bool((got[42:60] == 0).all())   # positions below 0, pages 7, 4, ...
    # row offsets that make no sense stay inside the buffers
    wq.wq_kv_write(x, x, cache, table, lens, cu_q=i32([-7, 2 ** 31 - 1, 3, 100]))
    wq.wq_kv_read(cache, table, i32([-3, 5, 2 ** 31 - 1]), 64, cu_q=i32([50, 10, 64, -2 ** 31]), out=(k, v))
    torch.cuda.synchronize()


def test_lengths_past_the_table(wq):
    """Rows past the table have no place: they neither move nor touch the cached ones."""
    P = _kv.Problem([32], None, 1, 64, 64, 16, F16, 61)
    table = P.table[:, :2].contiguous().cuda()
    cache = P.empty(wq)
    wq.wq_kv_write(P.K[0].cuda(), P.V[0].cuda(), cache, table, i32([32]))
    before = cache.data.clone()
    x = torch.randn(3, 1, 64).half().cuda()
    for n in (35, 40, 2 ** 31 - 1):
        wq.wq_kv_write(x, x, cache, table, i32([n]))
        assert torch.equal(cache.data, before)
    # the last of three rows at positions 30, 31, 32
    wq.wq_kv_write(x, x, cache, table, i32([33]))
    k, v = wq.wq_kv_read(cache, table, i32([33]), 33)
    assert same_bits(k[:30], _kv.stored(P.K[0][:30], 64)) and same_bits(k[30:32], _kv.stored(x[:2].cpu(), 64))
    assert float(k[32].abs().max()) == 0 and float(v[32].abs().max()) == 0
    # such a row still sees what is there
    q = torch.randn(1, 2, 64).half()
    K, V = torch.cat([P.K[0][:30], x[:2].cpu()]), torch.cat([P.V[0][:30], x[:2].cpu()])
    for n in (33, 50):
        out = wq.wq_kv_attention(q.cuda(), cache, table, i32([n]), window=40).cpu()
        want, bound = _kv.attention(q, K, V, torch.tensor([n - 1]), 0.125, True, 40, 64)
        assert bool(((out.double() - want).abs() <= bound).all())


def test_empty_calls(wq):
    cache = wq.wq_kv_cache(1, 16, 1, 64, 64, F16)
    x = torch.empty(0, 1, 64, dtype=F16, device="cuda")
    t = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    wq.wq_kv_write(x, x, cache, t, i32([]))
    k, v = wq.wq_kv_read(cache, t, i32([]), 0)
    assert k.shape == (0, 1, 64)
    assert wq.wq_kv_attention(x, cache, t, i32([])).shape == (0, 1, 64)
    # a table without pages: every row is without a place
    q = torch.ones(2, 1, 64, dtype=F16, device="cuda")
    t = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    wq.wq_kv_write(q, q, cache, t, i32([4, 4]))
    k, v = wq.wq_kv_read(cache, t, i32([4, 4]), 2)
    assert float(k.abs().max()) == 0 and float(v.abs().max()) == 0
    assert float(wq.wq_kv_attention(q, cache, t, i32([4, 4])).abs().max()) == 0


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def check_attention(wq, P, Hq, causal=True, window=0, ragged=None, scale=None, max_kv=None, q=None):
    cache = P.empty(wq)
    P.fill(wq, cache)
    if q is None:
        q = P.queries(Hq)
    scale = scale or P.D ** -0.5
    ragged = len(set(P.new)) > 1 if ragged is None else ragged
    out = wq.wq_kv_attention(q.cuda(), cache, P.table.cuda(), i32(P.lens), cu_q=P.cu(P.new).cuda() if ragged else None,
                             scale=scale, causal=causal, window=window, max_kv_len=max_kv)
    want, bound = P.reference(q, scale, causal, window)
    err = (out.cpu().double() - want).abs()
    worst = float((err / bound).max()) if err.numel() else 0.0
    assert bool((err <= bound).all()), f"error {float(err.max()):.3e}, {worst:.2f} of the bound"
    return out


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("D,G", SHAPES)
def test_attention_every_shape(wq, D, G, dt):
    """One token, a few and many rows per sequence (the two forms and their widths)."""
    for lens, new, Hq in (([1, 90, 64, 333], [1] * 4, 4), ([9, 150], [9, 5], 4), ([130, 77], [100, 77], 4)):
        check_attention(wq, _kv.Problem(lens, new, 2, D, G, 16, dt, D * 3 + G + len(new)), Hq)


@pytest.mark.parametrize("heads,kv", [(1, 1), (5, 5), (3, 1), (16, 1), (10, 2), (40, 2), (71, 1), (8, 8)])
def test_attention_head_layouts(wq, heads, kv):
    check_attention(wq, _kv.Problem([100, 41], [1, 1], kv, 64, 64, 32, F16, heads), heads)
    check_attention(wq, _kv.Problem([100, 41], [30, 7], kv, 64, 64, 32, F16, heads + 1), heads)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1023, 1024, 1025, 1031])
def test_attention_lengths(wq, n):
    check_attention(wq, _kv.Problem([n], [1], 1, 128, 128, 16, F16, n), 4)


@pytest.mark.parametrize("new", [1, 2, 16, 33, 64, 65, 129, 200])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 50), (False, 70), (True, 10 ** 6)])
def test_attention_masks(wq, new, causal, window):
    check_attention(wq, _kv.Problem([200, 260], [new, new], 1, 64, 32, 16, BF16, new), 2, causal, window)


def test_attention_sizes_past_32_bits(wq):
    """A window or an expected length that no 32-bit count holds means all there is."""
    P = _kv.Problem([100], [3], 1, 64, 64, 16, F16, 8)
    cache = P.empty(wq)
    P.fill(wq, cache)
    q = P.queries(2).cuda()
    args = (q, cache, P.table.cuda(), i32([100]))
    want = wq.wq_kv_attention(*args)
    for n in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 40):
        assert same_bits(wq.wq_kv_attention(*args, window=n), want)
        got = wq.wq_kv_attention(*args, max_kv_len=n).cpu().double()
        ref, bound = P.reference(q.cpu(), 0.125)
        assert bool(((got - ref).abs() <= bound).all())


@pytest.mark.parametrize("D,G,dt", [(128, 128, F16), (128, 64, BF16), (64, 32, F16), (256, 64, BF16)])
def test_attention_long_context_in_parts(wq, D, G, dt):
    """Few rows over many keys: the keys are split over workgroups and joined."""
    P = _kv.Problem([5003, 700], [1, 1], 1, D, G, 64, dt, D)
    assert wq.wq_kv_workspace_bytes(2, 2, False, 4, 1, D, G, 5003) > 0
    check_attention(wq, P, 4)
    check_attention(wq, P, 4, window=1500, max_kv=5003)
    P = _kv.Problem([2100, 64], [40, 64], 1, D, G, 64, dt, D)
    assert wq.wq_kv_workspace_bytes(104, 2, True, 4, 1, D, G, 2100) > 0
    check_attention(wq, P, 4)


@pytest.mark.parametrize("D,G,dt", [(128, 64, F16), (96, 32, BF16), (256, 128, F16)])
def test_attention_many_rows_in_few_parts(wq, D, G, dt):
    """Thousands of (row, head) outputs joined from a few parts, among them rows that some parts hold no key for and
    rows of no sequence."""
    P = _kv.Problem([1900, 550], [300, 250], 1, D, G, 32, dt, D + 1)
    per = wq.wq_kv_workspace_bytes(560, 2, True, 4, 1, D, G, 1900) // (560 * 4 * (D + 2) * 4)
    assert 2 <= per <= 8
    cache = P.empty(wq)
    P.fill(wq, cache)
    q = P.queries(4)
    wide = torch.zeros(560, 4, D, dtype=dt)
    wide[5:555] = q
    out = torch.full((560, 4, D), 2.0, dtype=dt, device="cuda")
    wq.wq_kv_attention(wide.cuda(), cache, P.table.cuda(), i32(P.lens), cu_q=i32([5, 305, 555]), window=700,
                       max_kv_len=1900, out=out)
    want, bound = P.reference(q, D ** -0.5, True, 700)
    got = out.cpu().double()
    assert bool(((got[5:555] - want).abs() <= bound).all())
    assert bool((got[:5] == 2).all()) and bool((got[555:] == 2).all())


@pytest.mark.parametrize("max_kv", [0, 1, 64, 5000, 10 ** 8])
def test_attention_any_expected_length(wq, max_kv):
    """max_kv_len shapes the launch and changes no result beyond the order of sums."""
    check_attention(wq, _kv.Problem([900, 3, 444], [1, 1, 1], 2, 128, 128, 16, F16, 9), 4, max_kv=max_kv)


def test_attention_ragged_many(wq):
    """More sequences than lanes, some without rows, some without tokens."""
    lens = [(13 * b) % 97 for b in range(150)]
    new = [min((b * 5) % 7, n) for b, n in enumerate(lens)]
    check_attention(wq, _kv.Problem(lens, new, 1, 64, 64, 16, F16, 3), 3)
    new = [min(b % 2 * (1 + b // 2), n) for b, n in enumerate(lens)]
    check_attention(wq, _kv.Problem(lens, new, 1, 64, 64, 16, F16, 4), 8)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("scale", [1e-3, 30.0])
def test_attention_value_ranges(wq, dt, scale):
    """Small and large values, flat and peaked rows, and rows of very unlike sizes."""
    P = _kv.Problem([300], [20], 1, 64, 32, 16, dt, 11, scale=scale)
    P.V[0][::7] *= 1 / 256
    P.V[0][150:] *= 64
    q = P.queries(2)
    q[3] *= 1e-4
    q[5] *= 4 / scale
    q[6] = 0
    check_attention(wq, P, 2, q=q)


def test_attention_growing_values(wq):
    """Value steps that grow by 2^30 along the keys move the reference of the sums again and again."""
    P = _kv.Problem([640], [1], 1, 64, 64, 16, BF16, 12)
    P.V[0] = (P.V[0].float() * torch.exp2(torch.arange(640) / 640 * 30 - 15)[:, None, None]).to(BF16)
    check_attention(wq, P, 2)
    P.V[0] = P.V[0].flip(0).contiguous()
    check_attention(wq, P, 2)


def test_attention_rows_that_see_nothing(wq):
    """Length 0, lengths below the rows, missing pages: zero, also in the joined form; rows of no sequence stay."""
    H, D = 1, 128
    P = _kv.Problem([64], [64], H, D, 128, 16, F16, 2)
    cache = P.empty(wq)
    P.fill(wq, cache)
    table = torch.cat([P.table[:, :4], torch.full((1, 4), -1, dtype=torch.int32)]).cuda()
    q = torch.randn(8, 2, D).half().cuda()
    for max_kv in (64, 100000):
        out = torch.full((8, 2, D), 3.0, dtype=F16, device="cuda")
        wq.wq_kv_attention(q, cache, table, i32([2, 64]), cu_q=i32([1, 5, 7]), out=out, max_kv_len=max_kv)
        got = out.cpu()
        assert bool((got[0] == 3).all()) and bool((got[7] == 3).all())
        assert bool((got[1:3] == 0).all()) and bool((got[5:7] == 0).all())  # rows at positions -2, -1; no pages
        want, bound = _kv.attention(q[3:5].cpu(), P.K[0][:2], P.V[0][:2], torch.tensor([0, 1]), D ** -0.5, True, 0, 128)
        assert bool(((got[3:5].double() - want).abs() <= bound).all())
    out = wq.wq_kv_attention(q, cache, i32([[0]] * 8), i32([0] * 8))
    assert float(out.abs().max()) == 0
    # all rows behind the last sequence
    out = torch.full((8, 2, D), 3.0, dtype=F16, device="cuda")
    wq.wq_kv_attention(q, cache, table, i32([64, 64]), cu_q=i32([0, 0, 0]), out=out, max_kv_len=100000)
    assert bool((out == 3).all())


def test_attention_hidden_places_hold_anything(wq):
    """NaN and infinities in keys and values past the mask, behind the window and in unwritten memory."""
    for new, window in ((1, 0), (40, 0), (40, 30), (1, 30)):
        P = _kv.Problem([200], [new], 1, 64, 64, 32, F16, new + window)
        cache = P.empty(wq)
        K, V = P.K[0].clone(), P.V[0].clone()
        if window:
            P.K[0][:131] = math.inf  # the first row's window begins at 131, inside a block of keys
            P.V[0][:131] = math.nan
        P.fill(wq, cache)
        # every row of the first query's future is NaN: only rows that see it may be
        q = P.queries(2)
        P.K[0], P.V[0] = K, V
        want, bound = P.reference(q, 0.125, True, window)
        out = wq.wq_kv_attention(q.cuda(), cache, P.table.cuda(), i32([200]), scale=0.125, window=window)
        err = (out.cpu().double() - want).abs()
        assert bool((err <= bound).all())
        if new > 1:  # poison the last token: only the last row sees it
            bad = torch.full((1, 1, 64), math.nan, dtype=F16, device="cuda")
            wq.wq_kv_write(bad, bad, cache, P.table.cuda(), i32([200]))
            out = wq.wq_kv_attention(q.cuda(), cache, P.table.cuda(), i32([200]), scale=0.125, window=window).cpu()
            assert bool(((out[:-1].double() - want[:-1]).abs() <= bound[:-1]).all())
            assert bool(out[-1].isnan().all())


def test_attention_nan_queries_stay_in_their_rows(wq):
    P = _kv.Problem([150], [40], 1, 64, 64, 16, F16, 21)
    q = P.queries(2)
    q[7, 1, 3] = math.nan
    q[9, 0, 0] = math.inf
    cache = P.empty(wq)
    P.fill(wq, cache)
    out = wq.wq_kv_attention(q.cuda(), cache, P.table.cuda(), i32([150])).cpu()
    assert bool(out[7, 1].isnan().all()) and bool(out[9, 0].isnan().all())
    q[7, 1] = 0
    q[9, 0] = 0
    want, bound = P.reference(q, 0.125)
    ok = (out.double() - want).abs() <= bound
    ok[7, 1] = ok[9, 0] = True
    assert bool(ok.all())


@pytest.mark.parametrize("dt", [F16, torch.bfloat16])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([20], [3]), ([70], [40])])
def test_attention_infinite_queries_are_nan(wq, dt, lens, new):
    """An infinite channel of a query whose keys all have the same sign there: every score is the same infinity, and
    the softmax of that is NaN; a row of the same call without a position stays zero."""
    P = _kv.Problem(lens, new, 1, 64, 64, 16, dt, 77)
    P.K[0].abs_().add_(1)
    cache = P.empty(wq)
    P.fill(wq, cache)
    for sign in (math.inf, -math.inf):
        q = P.queries(2)
        q[:, 0, 5] = sign
        q[-1, 0] = P.queries(2)[-1, 0]
        q[-1, 1, 63] = sign
        out = wq.wq_kv_attention(q.cuda(), cache, P.table.cuda(), i32(lens)).cpu()
        bad = q.isinf().any(-1)
        assert bool(out[bad].isnan().all()) and bool(out[~bad].isfinite().all())
        none = wq.wq_kv_attention(q.cuda(), cache, P.table.cuda(), i32([0])).cpu()
        assert bool((none == 0).all())


def test_attention_in_place(wq):
    """out may be q itself, in every form."""
    for lens, new, max_kv in (([70], [1], None), ([3000], [1], None), ([300], [80], None), ([90, 200], [1, 9], 100000)):
        P = _kv.Problem(lens, new, 1, 128, 128, 16, F16, 71)
        cache = P.empty(wq)
        P.fill(wq, cache)
        q = P.queries(4).cuda()
        args = (cache, P.table.cuda(), i32(lens))
        cu = P.cu(new).cuda()
        want = wq.wq_kv_attention(q, *args, cu_q=cu, max_kv_len=max_kv)
        got = wq.wq_kv_attention(q, *args, cu_q=cu, max_kv_len=max_kv, out=q)
        assert got.data_ptr() == q.data_ptr() and same_bits(got, want)


def test_attention_strided(wq):
    P = _kv.Problem([90, 33], [1, 1], 2, 128, 128, 16, F16, 31)
    cache = P.empty(wq)
    P.fill(wq, cache)
    wide = torch.randn(2, 12 * 128).half().cuda()
    q = wide[:, 2 * 128:6 * 128].view(2, 4, 128)
    o = torch.full((2, 6 * 128), 9.0, dtype=F16, device="cuda")
    out = o[:, 128:5 * 128].view(2, 4, 128)
    wq.wq_kv_attention(q, cache, P.table.cuda(), i32(P.lens), out=out)
    want, bound = P.reference(q.cpu().contiguous(), 128 ** -0.5)
    assert bool(((out.cpu().double() - want).abs() <= bound).all())
    assert bool((o[:, :128] == 9).all()) and bool((o[:, 5 * 128:] == 9).all())


@pytest.mark.parametrize("lens,new,max_kv", [([90, 33], [1, 1], None), ([300], [80], None), ([3000], [1], None)])
def test_attention_beside_its_queries(wq, lens, new, max_kv):
    """Queries and outputs as slices of one buffer's rows, either first; over each other they are refused."""
    P = _kv.Problem(lens, new, 2, 64, 64, 16, F16, 32)
    cache = P.empty(wq)
    P.fill(wq, cache)
    q = P.queries(4)
    want, bound = P.reference(q, 0.125)
    for at_q, at_o in ((0, 4), (4, 0)):
        wide = torch.full((sum(new), 8, 64), 9.0, dtype=F16, device="cuda")
        wide[:, at_q:at_q + 4] = q.cuda()
        out = wide[:, at_o:at_o + 4]
        wq.wq_kv_attention(wide[:, at_q:at_q + 4], cache, P.table.cuda(), i32(lens), out=out, max_kv_len=max_kv)
        assert bool(((out.cpu().double() - want).abs() <= bound).all())
        assert torch.equal(wide[:, at_q:at_q + 4].cpu(), q)
        with pytest.raises(wq.WQError) as e:
            wq.wq_kv_attention(wide[:, 1:5], cache, P.table.cuda(), i32(lens), out=wide[:, 2:6], max_kv_len=max_kv)
        assert e.value.status == 1
    k = torch.zeros(sum(new), 2, 64, dtype=F16, device="cuda")
    with pytest.raises(wq.WQError) as e:
        wq.wq_kv_read(cache, P.table.cuda(), i32(lens), sum(new), out=(k, k))
    assert e.value.status == 1


def test_attention_of_rotated_rows(wq):
    """Queries and keys rotated head by head (wq_hadamard) before they are cached: the same attention, with an outlier
    channel spread over its group."""
    H, D, n = 2, 128, 150
    P = _kv.Problem([n], [5], H, D, 128, 16, F16, 91)
    P.K[0][:, :, 17] *= 12
    q = P.queries(4)
    a = torch.softmax(q[:, 0].double() @ P.K[0][:, 0].double().T * 0.05 + torch.full((5, n), 0.0).masked_fill(
        torch.arange(n)[None] > torch.arange(n - 5, n)[:, None], -math.inf).double(), 1) @ P.V[0][:, 0].double()
    rot = lambda x: wq.wq_hadamard(x.reshape(-1, D).cuda(), D).view(x.shape)
    errors = []
    for turn in (lambda x: x.cuda(), rot):
        kq, kk = turn(q), turn(P.K[0])
        cache = wq.wq_kv_cache(P.num_pages, 16, H, D, 128, F16)
        wq.wq_kv_write(kk, P.V[0].cuda(), cache, P.table.cuda(), i32([n]))
        out = wq.wq_kv_attention(kq, cache, P.table.cuda(), i32([n]), scale=0.05).cpu()
        want, bound = _kv.attention(kq.cpu(), kk.cpu(), P.V[0], torch.arange(n - 5, n), 0.05, True, 0, 128)
        assert bool(((out.double() - want).abs() <= bound).all())
        errors.append(float((out[:, 0].double() - a).norm() / a.norm()))
    assert errors[1] < errors[0]  # the rotated keys lose less to 4 bits


def test_cache_beyond_4_gib(wq):
    """Pages whose bytes lie past 32-bit offsets."""
    H, D, page = 8, 128, 1024
    pages = (5 << 30) // (H * page // 16 * (16 * D + 128)) + 1
    cache = wq.wq_kv_cache(pages, page, H, D, 128, F16)
    P = _kv.Problem([1100], [1], H, D, 128, page, F16, 41)
    P.table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32)
    P.num_pages = pages
    P.fill(wq, cache)
    k, v = read_all(wq, P, cache)
    assert same_bits(k, _kv.stored(P.K[0], 128)) and same_bits(v, _kv.stored(P.V[0], 128))
    q = P.queries(8)
    out = wq.wq_kv_attention(q.cuda(), cache, P.table.cuda(), i32([1100]))
    want, bound = P.reference(q, 128 ** -0.5)
    assert bool(((out.cpu().double() - want).abs() <= bound).all())


# ---------------------------------------------------------------------------
# Streams and graphs
# ---------------------------------------------------------------------------
def test_streams_and_graph(wq):
    """A decode step (write, attend) captured once and replayed as the lengths grow, on a stream of its own, against
    the eager calls; two attention calls share one workspace."""
    H, D, Hq, T = 2, 128, 8, 1300
    P = _kv.Problem([T, T - 300], [1, 1], H, D, 128, 16, F16, 51)
    table = P.table.cuda()
    need = wq.wq_kv_workspace_bytes(2, 2, False, Hq, H, D, 128, T)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    start = [T - 6, T - 306]
    Q = torch.randn(6, 2, Hq, D).half()

    def history(cache):
        k = torch.cat([P.K[b][:start[b]] for b in range(2)]).cuda()
        v = torch.cat([P.V[b][:start[b]] for b in range(2)]).cuda()
        wq.wq_kv_write(k, v, cache, table, i32(start), cu_q=P.cu(start).cuda())

    eager_cache, cache = P.empty(wq), P.empty(wq)
    history(eager_cache)
    history(cache)
    eager = []
    rows = [(torch.stack([P.K[b][start[b] + i] for b in range(2)]).cuda(),
             torch.stack([P.V[b][start[b] + i] for b in range(2)]).cuda()) for i in range(6)]
    for i in range(6):
        lens = i32([s + i + 1 for s in start])
        wq.wq_kv_write(*rows[i], eager_cache, table, lens)
        eager.append(wq.wq_kv_attention(Q[i].cuda(), eager_cache, table, lens, max_kv_len=T, ws=ws).clone())
    k, v, q, lens = rows[0][0].clone(), rows[0][1].clone(), Q[0].cuda(), i32([s + 1 for s in start])
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        wq.wq_kv_write(k, v, cache, table, lens)
        wq.wq_kv_attention(q, cache, table, lens, max_kv_len=T, out=out, ws=ws)
        wq.wq_kv_attention(q, cache, table, lens, max_kv_len=T, out=out2, ws=ws)
    for i in range(6):
        k.copy_(rows[i][0])
        v.copy_(rows[i][1])
        q.copy_(Q[i])
        lens.copy_(i32([s + i + 1 for s in start]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(out, eager[i]) and same_bits(out2, eager[i]), i
    # an explicit stream
    side.wait_stream(torch.cuda.current_stream())
    got = wq.wq_kv_attention(q, cache, table, lens, max_kv_len=T, ws=ws, out=torch.empty_like(q), stream=side)
    side.synchronize()
    assert same_bits(got, eager[5])
