"""Norm, rotary positions, adapters and page tables on the GPU against their references in 64 bits (tests/_layer.py,
which derives the bounds)."""
import math
import random

import pytest
import torch

import _layer
import weight_only_quantized_w4a16_amd as wq

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16]
i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()


@pytest.fixture(scope="module", autouse=True)
def gpu():
    wq.lib()
    assert torch.cuda.is_available()


def within(got, want, bound, what=""):
    err = (got.detach().cpu().double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((err - bound)[bad].max()), float(err.max()))


def randn(g, *shape):
    return torch.randn(shape, generator=g)


# ---------------------------------------------------------------------------- norm
NORM_DIMS = [8, 16, 64, 72, 128, 256, 264, 512, 520, 1000, 2048, 2056, 4096, 5000, 8192, 8200, 16384, 20000, 32768, 65536]


@pytest.mark.parametrize("dim", NORM_DIMS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_norm(dim, dtype):
    g = torch.Generator().manual_seed(dim)
    for rows in (1, 3, 67, 300 if dim <= 2056 else 33):
        x, r = (randn(g, rows, dim) * (1 + 20 * (torch.rand(dim, generator=g) < 0.02)) for _ in range(2))
        x, r, w = x.to(dtype), r.to(dtype), (1 + 0.3 * randn(g, dim)).to(dtype)
        y, yb, _, _ = _layer.rms_norm(x, w, 1e-5)
        within(wq.wq_rms_norm(x.cuda(), w.cuda(), 1e-5), y, yb, rows)
        y, yb, h, hb = _layer.rms_norm(x, w, 1e-6, r)
        got, s = wq.wq_rms_norm(x.cuda(), w.cuda(), residual=r.cuda())
        within(got, y, yb, rows)
        within(s, h, hb, rows)
        # every place an output may take
        for out, sum_out in (("x", "r"), ("r", "x"), ("x", None), (None, "x"), (None, "r"), ("r", None)):
            t = dict(x=x.cuda(), r=r.cuda())
            a, b = wq.wq_rms_norm(t["x"], w.cuda(), residual=t["r"], out=t.get(out), sum_out=t.get(sum_out))
            assert torch.equal(a, got) and torch.equal(b, s), (out, sum_out)
        t = x.cuda()
        assert torch.equal(wq.wq_rms_norm(t, w.cuda(), 1e-5, out=t), wq.wq_rms_norm(x.cuda(), w.cuda(), 1e-5))


@pytest.mark.parametrize("heads,dim", [(1, 64), (7, 64), (32, 128), (5, 80), (3, 256), (2, 4096), (40, 96)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_of_heads_in_a_projection(heads, dim, dtype):
    g = torch.Generator().manual_seed(heads * dim)
    for rows in (1, 2, 41):
        qkv = randn(g, rows, heads + 3, dim).to(dtype)
        w = (1 + 0.3 * randn(g, dim)).to(dtype)
        buf = qkv.cuda()
        y, yb, _, _ = _layer.rms_norm(qkv[:, 1:heads + 1], w, 1e-6)
        got = wq.wq_rms_norm(buf[:, 1:heads + 1], w.cuda(), 1e-6)
        assert got.is_contiguous()
        within(got, y, yb)
        assert wq.wq_rms_norm(buf[:, 1:heads + 1], w.cuda(), 1e-6, out=buf[:, 1:heads + 1]) is not None  # in place
        assert torch.equal(buf[:, 1:heads + 1], got)
        assert torch.equal(buf[:, 0].cpu(), qkv[:, 0]) and torch.equal(buf[:, heads + 1:].cpu(), qkv[:, heads + 1:])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 4096])
def test_norm_of_unusual_values(dtype, dim):
    g = torch.Generator().manual_seed(5)
    x, w = randn(g, 9, dim).to(dtype), torch.ones(dim).to(dtype)
    x[1], x[3, 7], x[5, 1], x[6], x[7] = 0, math.inf, math.nan, 6e4, 2.0 ** -20
    got = wq.wq_rms_norm(x.cuda(), w.cuda(), 1e-6).cpu()
    assert torch.equal(got[1], torch.zeros(dim).to(dtype))
    assert got[3, 7].isnan() and not got[3, :7].any() and not got[3, 8:].any()
    assert got[5].isnan().all()
    keep = [0, 2, 4, 6, 7, 8]
    y, yb, _, _ = _layer.rms_norm(x[keep], w, 1e-6)
    within(got[keep], y, yb)
    assert wq.wq_rms_norm(x[:0].cuda(), w.cuda()).shape == (0, dim)


def test_norm_between_the_rows_of_its_input():
    g = torch.Generator().manual_seed(6)
    x, w = randn(g, 5, 256).half(), torch.ones(128).half()
    buf = x.cuda()
    wq.wq_rms_norm(buf[:, :128], w.cuda(), out=buf[:, 128:])
    y, yb, _, _ = _layer.rms_norm(x[:, :128], w, 1e-6)
    within(buf[:, 128:], y, yb)
    assert torch.equal(buf[:, :128].cpu(), x[:, :128])


# ---------------------------------------------------------------------------- rotary positions
def plan_of(D, R, axes, adjacent, base=10000.0, factor=1.0):
    half = R // 2
    axis = [i * axes // half for i in range(half)] if axes > 1 else [0] * half
    p = wq.wq_rotary_plan(D, R, base=base, axes=axis if axes > 1 else None, adjacent=adjacent, factor=factor)
    return p, [base ** (-2.0 * i / R) for i in range(half)], axis


@pytest.mark.parametrize("D,R", [(64, 64), (80, 80), (96, 32), (128, 128), (128, 64), (256, 64), (192, 192), (512, 512), (16, 16)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rotary_positions(D, R, adjacent, dtype):
    g = torch.Generator().manual_seed(D + R)
    for T, Hq, Hk, axes in ((1, 8, 1, 1), (5, 1, 1, 3), (70, 5, 2, 1), (33, 32, 8, 2)):
        plan, freqs, axis = plan_of(D, R, axes, adjacent, factor=1.25)
        qkv = randn(g, T, Hq + 2 * Hk, D).to(dtype)
        pos = torch.randint(-3, 1 << 20, (axes, T), generator=g).to(torch.int32)
        q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        buf = qkv.cuda()
        qd, kd = buf[:, :Hq], buf[:, Hq:Hq + Hk]
        given = pos[0].cuda() if axes == 1 else pos.cuda()
        a, b = wq.wq_rotary(qd, kd, plan, positions=given)
        want_q, bound_q = _layer.rotary(q, pos, freqs, axis, adjacent, 1.25)
        want_k, bound_k = _layer.rotary(k, pos, freqs, axis, adjacent, 1.25)
        within(a, want_q, bound_q)
        within(b, want_k, bound_k)
        assert torch.equal(buf.cpu(), qkv)
        one, none = wq.wq_rotary(qd, None, plan, positions=given)
        assert none is None and torch.equal(one, a)
        wq.wq_rotary(qd, kd, plan, positions=given, out=(qd, kd))  # in place
        assert torch.equal(qd, a) and torch.equal(kd, b) and torch.equal(buf[:, Hq + Hk:].cpu(), qkv[:, Hq + Hk:])


@pytest.mark.parametrize("new,total", [([1] * 5, [1, 131072, 77, 999999, 3]), ([7, 1, 0, 30, 64, 1], [7, 100, 5, 30, 70000, 64]),
                                       ([300], [300]), ([0, 0, 3], [4, 5, 6]), ([1] * 200, list(range(1, 201)))])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rotary_of_sequences(new, total, dtype):
    """Positions from the lengths; rows outside every sequence stay as they were."""
    g = torch.Generator().manual_seed(len(new))
    plan, freqs, axis = plan_of(128, 128, 3, False, 500000.0)
    cu, at = [2], []
    for q, n in zip(new, total):
        cu.append(cu[-1] + q)
        at += range(n - q, n)
    T = cu[-1] + 3
    q, k = randn(g, T, 8, 128).to(dtype), randn(g, T, 2, 128).to(dtype)
    a, b = q.cuda(), k.cuda()
    wq.wq_rotary(a, b, plan, kv_lens=i32(total), cu_q=i32(cu), out=(a, b))
    pos = torch.tensor(at)[None].expand(3, -1)
    for x, y in ((q, a), (k, b)):
        want, bound = _layer.rotary(x[2:-3], pos, freqs, axis, False, 1.0)
        within(y[2:-3], want, bound)
        assert torch.equal(y[:2].cpu(), x[:2]) and torch.equal(y[-3:].cpu(), x[-3:])
    if len(set(new)) == 1 and new[0]:  # the same without offsets
        c, d = wq.wq_rotary(q[2:-3].cuda(), k[2:-3].cuda(), plan, kv_lens=i32(total))
        assert torch.equal(c, a[2:-3]) and torch.equal(d, b[2:-3])


def test_rotary_of_far_positions():
    """Positions near 2^31 keep their angle: the same as a near position a whole number of turns before."""
    half = 32
    plan = wq.wq_rotary_plan(64, freqs=[2 * math.pi * (i + 1) / 128 for i in range(half)])
    g = torch.Generator().manual_seed(3)
    x = randn(g, 4, 3, 64).half().cuda()
    near = i32([5, 127, -128, 0])
    far = i32([5 + 128 * (1 << 23), 127 + 128 * 16000000, -128 - 128 * (1 << 23), -2147483648])
    a, _ = wq.wq_rotary(x, None, plan, positions=near)
    b, _ = wq.wq_rotary(x, None, plan, positions=far)
    # the frequency is held to 2^-54 of a turn: 2^-23 at 2^31 positions
    assert float((a.double() - b.double()).abs().max()) <= 2 * math.pi * 2.0 ** -22 * float(x.abs().max()) * 2 + 2.0 ** -9


# ---------------------------------------------------------------------------- adapters
def adapters_case(g, dtype, new, K, slices, rank, num, mixed, lead=0, tail=0, junk=False):
    cu = [lead]
    for q in new:
        cu.append(cu[-1] + q)
    T, S, N = cu[-1] + tail, len(slices), sum(slices)
    x, y = randn(g, T, K).to(dtype), randn(g, T, N).mul(2).to(dtype)
    a, b = (randn(g, num, S, rank, K) / math.sqrt(K)).to(dtype), (randn(g, num, N, rank) * 0.5).to(dtype)
    ids = [int(v) for v in torch.randint(-1, num + (1 if len(new) > 4 else 0), (len(new),), generator=g)]
    ids[0] = num - 1
    ranks = [int(v) for v in torch.randint(0, rank + 1, (num,), generator=g)] if mixed else [rank] * num
    if mixed:
        ranks[num - 1] = max(1, ranks[num - 1])
    scales = torch.rand(num, generator=g) * 3 - 0.5
    if junk:  # what lies past a rank is not used
        for i, r in enumerate(ranks):
            a[i, :, r:], b[i, :, r:] = math.nan, math.inf
    bank = wq.LoraBank(a.cuda(), b.cuda(), scales.cuda(), i32(ranks) if mixed else None, tuple(slices))
    row_ids = [-1] * lead + [i for i, q in zip(ids, new) for _ in range(q)] + [-1] * tail
    if junk:
        a, b = a.nan_to_num(0.0), b.nan_to_num(0.0, 0.0, 0.0)
    want, bound = _layer.lora(x, y, a, b, scales, ranks, slices, row_ids)
    return dict(x=x, y=y, bank=bank, ids=ids, cu=cu, want=want, bound=bound, T=T, N=N)


LORA = [([1], 128, [16], 8, 1, False), ([1], 4096, [4096], 16, 8, False), ([1] * 17, 512, [256, 64, 64], 16, 5, True),
        ([1] * 64, 1152, [1008], 32, 40, True), ([3] * 11, 256, [48], 24, 3, True), ([40], 384, [272, 16], 64, 2, False),
        ([100, 1, 0, 33, 64, 7], 640, [128, 128, 128], 64, 4, False), ([130, 200], 1024, [512], 128, 3, True),
        ([16] * 16, 256, [32, 16, 16, 64], 8, 7, True), ([70], 128, [4112], 128, 1, False), ([1] * 130, 256, [144], 40, 200, True),
        ([500, 3], 2176, [80], 16, 2, False),
        # many rows: several blocks of columns to a workgroup, several parts of K
        ([700, 600], 128, [16384], 64, 2, False), ([651, 1, 649], 1152, [8192, 8192], 16, 3, True),
        ([1290], 128, [15984, 400], 128, 1, False),
        # many short sequences: many adapters to a tile of rows
        ([1] * 300, 1152, [208, 32], 16, 40, True), ([2] * 170, 640, [96], 24, 100, False), ([1] * 1100, 256, [80, 48], 16, 90, True),
        ([3] * 400, 1152, [64], 64, 7, True), ([1] * 700 + [900], 256, [144], 32, 2, False),
        # few rows of one or two sequences: several items of an adapter
        ([16], 640, [272], 16, 3, False), ([9, 4], 384, [96, 32], 24, 2, True), ([64], 1152, [528], 32, 2, False),
        ([90, 38], 256, [64], 128, 3, True), ([250], 1024, [144, 48], 16, 2, False), ([5] * 50, 384, [96], 40, 30, True)]


@pytest.mark.parametrize("case", LORA, ids=[f"{sum(c[0])}x{c[1]}-r{c[3]}" for c in LORA])
@pytest.mark.parametrize("dtype", DTYPES)
def test_adapters(case, dtype):
    new, K, slices, rank, num, mixed = case
    g = torch.Generator().manual_seed(sum(new) + K)
    c = adapters_case(g, dtype, new, K, slices, rank, num, mixed)
    x, y, ids = c["x"].cuda(), c["y"].cuda(), i32(c["ids"])
    even = len(set(new)) == 1
    got = wq.wq_lora(x, c["bank"], ids, y, cu_q=None if even else i32(c["cu"]))
    within(got, c["want"], c["bound"])
    assert torch.equal(y.cpu(), c["y"])
    for _ in range(4):  # offsets say the same; the same bits every time
        assert torch.equal(wq.wq_lora(x, c["bank"], ids, y, cu_q=i32(c["cu"])), got)
    need = wq.wq_lora_workspace_bytes(c["T"], len(new), K, rank, len(slices))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever it is read before it is written
    wq.wq_lora(x, c["bank"], ids, y, cu_q=i32(c["cu"]), out=y, ws=ws)  # in place
    assert torch.equal(y, got)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lead,tail", [(0, 5), (3, 0), (17, 40)])
def test_adapters_leave_other_rows(dtype, lead, tail):
    g = torch.Generator().manual_seed(lead)
    c = adapters_case(g, dtype, [5, 0, 20, 1, 1, 30], 256, [96, 32], 16, 4, True, lead, tail, junk=True)
    x, y, ids, cu = c["x"].cuda(), c["y"].cuda(), i32(c["ids"]), i32(c["cu"])
    out = torch.full_like(y, 7)
    wq.wq_lora(x, c["bank"], ids, y, cu_q=cu, out=out)
    end = c["T"] - tail
    within(out[lead:end], c["want"][lead:end], c["bound"][lead:end])
    assert bool((out[:lead] == 7).all()) and bool((out[end:] == 7).all())
    for none in ([-1] * 6, [4] * 6, [-2147483648] * 6, [2147483647] * 6):
        out.fill_(7)
        wq.wq_lora(x, c["bank"], i32(none), y, cu_q=cu, out=out)
        assert torch.equal(out[lead:end], y[lead:end]) and bool((out[end:] == 7).all())
    for odd in ([0] * 7, [1 << 30] * 7, [-5, 3, 2, 9, 4, 1 << 30, 3]):  # offsets that are none: within the buffers
        wq.wq_lora(x, c["bank"], ids, y, cu_q=i32(odd), out=out)
        wq.wq_rotary(torch.zeros(c["T"], 1, 64, dtype=dtype, device="cuda"), None, wq.wq_rotary_plan(64), kv_lens=ids,
                     cu_q=i32(odd))
    assert wq.wq_lora(x[:0], c["bank"], ids[:0], y[:0]).shape == (0, c["N"])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [[1] + [0] * 100 + [1, 0, 2], [0] * 200 + [3] + [0] * 70, [200, 0, 150, 1, 40] + [0] * 80 + [5]])
def test_adapters_of_sequences_without_rows(dtype, new):
    """More empty sequences than a wave has lanes; few rows and many; in place and not, some without an adapter, an
    adapter of rank 0, junk past the ranks."""
    g = torch.Generator().manual_seed(len(new) + sum(new))
    c = adapters_case(g, dtype, new, 256, [96, 48], 24, 5, True, 2, 3, junk=True)
    x, y, ids, cu = c["x"].cuda(), c["y"].cuda(), i32(c["ids"]), i32(c["cu"])
    out = torch.full_like(y, 7)
    wq.wq_lora(x, c["bank"], ids, y, cu_q=cu, out=out)
    end = c["T"] - 3
    within(out[2:end], c["want"][2:end], c["bound"][2:end])
    assert bool((out[:2] == 7).all()) and bool((out[end:] == 7).all())
    wq.wq_lora(x, c["bank"], ids, y, cu_q=cu, out=y)
    assert torch.equal(y[2:end], out[2:end])
    plan = wq.wq_rotary_plan(64)
    q = randn(g, c["T"], 3, 64).to(dtype)
    lens = [n + 5 for n in new]
    turned = q.cuda()
    wq.wq_rotary(turned, None, plan, kv_lens=i32(lens), cu_q=cu, out=(turned, None))
    at = [p for n in new for p in range(5, 5 + n)]
    want, bound = _layer.rotary(q[2:end], torch.tensor([at]), [10000.0 ** (-i / 32) for i in range(32)], [0] * 32, False, 1.0)
    within(turned[2:end], want, bound)
    assert torch.equal(turned[:2].cpu(), q[:2]) and torch.equal(turned[end:].cpu(), q[end:])


def test_offsets_past_32_bits():
    """Matrices of more than 2^31 elements: the last rows come out as they do alone."""
    rows, width = 70000, 32768
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, width, dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 10000):
        x[i:i + 10000] = torch.randn(10000, width, generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(width, generator=g, device="cuda").bfloat16()
    tail = x[-50:].clone()
    assert torch.equal(wq.wq_rms_norm(x, w)[-50:], wq.wq_rms_norm(tail, w))
    plan = wq.wq_rotary_plan(128)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    a = wq.wq_rotary(x.view(rows, 256, 128), None, plan, positions=pos)[0][-50:]
    assert torch.equal(a, wq.wq_rotary(tail.view(50, 256, 128), None, plan, positions=pos[-50:])[0])
    bank = wq.LoraBank((torch.randn(2, 16, 256, generator=g, device="cuda") / 16).bfloat16(),
                       torch.randn(2, width, 16, generator=g, device="cuda").bfloat16(), torch.ones(2, device="cuda"))
    xs = torch.randn(rows, 256, generator=g, device="cuda").bfloat16()
    ids = i32([0, 1])
    got = wq.wq_lora(xs, bank, ids, x, cu_q=i32([0, rows - 50, rows]), out=x)[-50:]
    # (the tail alone is summed in another order: within its bound)
    want, bound = _layer.lora(xs[-50:].cpu(), tail.cpu(), bank.a.cpu()[:, None], bank.b.cpu(), [1.0, 1.0], [16, 16], (width,), [1] * 50)
    within(got, want, bound)


@pytest.mark.parametrize("dtype", DTYPES)
def test_adapters_of_large_and_infinite_values(dtype):
    """x A^T past fp16's range, an infinity in one row, a NaN in another: the other rows hold."""
    g = torch.Generator().manual_seed(9)
    c = adapters_case(g, dtype, [1] * 6, 256, [64], 16, 1, False)
    bank = c["bank"]
    x, y = c["x"].clone(), c["y"]
    x[1] *= 2000.0
    a = bank.a.cpu().clone() * 100
    x[2, 5], x[3, 9] = math.inf, math.nan
    ids = [0] * 6
    big = wq.LoraBank(a.cuda(), bank.b, bank.scales * 1e-4, slices=(64,))
    got = wq.wq_lora(x.cuda(), big, i32(ids), y.cuda()).cpu()
    keep = [0, 1, 4, 5]
    want, bound = _layer.lora(x[keep], y[keep], a, bank.b.cpu(), (bank.scales * 1e-4).cpu(), [16], [64], [0] * 4)
    within(got[keep], want, bound)
    assert float((x[1].double() @ a[0, 0].double().t()).abs().max()) > 65504
    assert not got[2].isfinite().any() and got[3].isnan().all()


# ---------------------------------------------------------------------------- page tables
def same(pages, ref, got, want):
    cu, pos, slots = want
    assert got[0].tolist() == cu and got[1].tolist() == pos and got[2].tolist() == slots
    assert pages.block_table.tolist() == ref.table and pages.kv_lens.tolist() == ref.lens
    assert pages.free.tolist() == ref.free and pages.counts.tolist() == [ref.count, ref.lack]


@pytest.mark.parametrize("batch,max_pages,num_pages,page", [(1, 4, 6, 16), (5, 9, 30, 32), (64, 20, 700, 16), (1500, 3, 3000, 16),
                                                            (3, 600, 1500, 64), (2, 5000, 9000, 16)])
def test_resize(batch, max_pages, num_pages, page):
    rng = random.Random(batch)
    pages = wq.wq_kv_pages(num_pages, page, batch, max_pages)
    ref = _layer.Pages([[-1] * max_pages for _ in range(batch)], [0] * batch, range(num_pages - 1, -1, -1), num_pages, page)
    cap = max_pages * page
    failed = 0
    for step in range(12):
        kind = rng.choice(["grow", "grow", "mixed", "shrink", "large", "beyond"])
        want = []
        for n in ref.lens:
            if kind == "grow":
                m = n + rng.randint(0, 9)
            elif kind == "shrink":
                m = max(0, n - rng.randint(0, 9))
            elif kind == "large":
                m = rng.randint(0, cap)
            else:
                m = rng.choice([0, n, rng.randint(0, min(cap, max(1, num_pages // batch) * page))])
            want.append(min(m, cap))
        if kind == "beyond":
            want[rng.randrange(batch)] = rng.choice([-1, cap + 1, 2147483647, -2147483648])
        new = sum(max(0, m - n) for n, m in zip(ref.lens, want)) if kind != "beyond" else 40
        rows = max(0, min(new, 200000) + rng.choice([0, 0, 7, -3]))
        expect = ref.resize(want, rows)
        failed += ref.lack != 0
        same(pages, ref, wq.wq_kv_resize(pages, i32(want), rows), expect)
    expect = ref.resize([0] * batch, 0)
    same(pages, ref, wq.wq_kv_resize(pages, i32([0] * batch)), expect)
    assert pages.counts.tolist() == [num_pages, 0] and sorted(ref.free) == list(range(num_pages))


def test_resize_takes_what_comes_back():
    """All pages in use: a sequence that ends feeds the others in the same call; one page too many changes nothing."""
    pages = wq.wq_kv_pages(8, 16, 3, 8)
    ref = _layer.Pages([[-1] * 8 for _ in range(3)], [0] * 3, range(7, -1, -1), 8, 16)
    for want in ([64, 64, 0], [0, 64, 64], [0, 65, 64], [16, 0, 112], [0, 0, 128], [1, 0, 128], [128, 0, 0]):
        expect = ref.resize(want, 30)
        same(pages, ref, wq.wq_kv_resize(pages, i32(want), 30), expect)
    # a state that gives back more pages than there are is not a change
    pages.counts[0] = 8
    before = pages.free.clone()
    cu, pos, slots = wq.wq_kv_resize(pages, i32([0, 0, 0]), 2)
    assert pages.counts.tolist() == [8, -1] and torch.equal(pages.free, before) and pages.kv_lens.tolist() == [128, 0, 0]
    assert not cu.any() and bool((pos == -1).all()) and bool((slots == -1).all())
    empty = wq.wq_kv_pages(4, 16, 0, 3)
    assert wq.wq_kv_resize(empty, i32([]), 2)[0].tolist() == [0] and empty.counts.tolist() == [4, 0]


@pytest.mark.parametrize("batch", [3, 1024, 1025])
def test_resize_of_many_rows(batch):
    """More rows than one workgroup takes: changes that fit, that lack pages and that have no place, eager and captured."""
    per = 24000 // batch
    cap = -(-per // 16) + 2
    num_pages = batch * (cap - 1)
    pages = wq.wq_kv_pages(num_pages, 16, batch, cap)
    ref = _layer.Pages([[-1] * cap for _ in range(batch)], [0] * batch, range(num_pages - 1, -1, -1), num_pages, 16)
    even, odd = [per if b % 2 == 0 else 0 for b in range(batch)], [per if b % 2 else 0 for b in range(batch)]
    changes = [even, [per + 16] * batch, odd, [per] * (batch - 1) + [16 * cap + 1], [16 * cap] * batch, even[::-1],
               [n - n % 5 for n in odd], [0] * batch]
    assert batch * cap > num_pages and sum(even) > 8192 and sum(odd) > 7000
    lacked = []
    for want in changes:
        expect = ref.resize(want, 20000)
        lacked.append(ref.lack)
        same(pages, ref, wq.wq_kv_resize(pages, i32(want), 20000), expect)
    assert lacked[3] == -1 and lacked[4] > 0 and lacked.count(0) == len(changes) - 2
    want = i32(changes[0])
    wq.wq_kv_resize(pages, want, 20000)  # (and back: the state that the graph is captured from)
    wq.wq_kv_resize(pages, i32([0] * batch))
    main = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        out = wq.wq_kv_resize(pages, want, 20000)
    ref.resize(changes[0], 20000), ref.resize(changes[-1], 0)
    for wanted in changes:
        want.copy_(i32(wanted))
        expect = ref.resize(wanted, 20000)
        graph.replay()
        torch.cuda.synchronize()
        same(pages, ref, out, expect)


# ---------------------------------------------------------------------------- streams and graphs
def test_calls_on_another_stream_and_in_a_graph():
    """Each operator on an explicit stream, and captured: every replay gives the eager results on new inputs."""
    g = torch.Generator().manual_seed(12)
    dt = torch.float16
    c = adapters_case(g, dt, [1] * 20, 512, [256, 128, 128], 16, 6, True)
    x, r, w = randn(g, 20, 512).to(dt).cuda(), randn(g, 20, 512).to(dt).cuda(), torch.ones(512, dtype=dt, device="cuda")
    y, ids = c["y"].cuda(), i32(c["ids"])
    q, k = randn(g, 20, 6, 64).to(dt).cuda(), randn(g, 20, 2, 64).to(dt).cuda()
    plan = wq.wq_rotary_plan(64)
    pages = wq.wq_kv_pages(200, 16, 20, 9)
    lens = i32([5] * 20)

    def step(stream=None):
        cu, pos, slots = wq.wq_kv_resize(pages, lens, 100, stream=stream)
        n, s = wq.wq_rms_norm(x, w, residual=r, stream=stream)
        o = wq.wq_lora(n, c["bank"], ids, y, stream=stream)
        a, b = wq.wq_rotary(q, k, plan, kv_lens=pages.kv_lens, stream=stream)
        return cu, pos, slots, n, s, o, a, b

    def reset():
        fresh = wq.wq_kv_pages(200, 16, 20, 9)
        for name in ("block_table", "kv_lens", "free", "counts"):
            getattr(pages, name).copy_(getattr(fresh, name))

    reset()
    want = [t.clone() for t in step()]
    reset()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = step(side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q_) for p, q_ in zip(want, got))
    reset()
    main = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        out = step()
    for i in range(4):
        gi = torch.Generator().manual_seed(100 + i)
        x.copy_(randn(gi, 20, 512)), y.copy_(randn(gi, 20, 512)), q.copy_(randn(gi, 20, 6, 64))
        lens.copy_(torch.randint(1, 90, (20,), generator=gi))
        ids.copy_(torch.randint(-1, 6, (20,), generator=gi))
        reset()
        want = [t.clone() for t in step()]
        reset()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for p, q_ in zip(want, out):
            assert torch.equal(p, q_), i


def test_two_streams_at_once():
    """Calls that overlap on two streams have scratch of their own."""
    g = torch.Generator().manual_seed(13)
    cases = [adapters_case(g, torch.bfloat16, [1] * 48, 2048, [1024], 32, 30, False) for _ in range(2)]
    xs, ys = [c["x"].cuda() for c in cases], [c["y"].cuda() for c in cases]
    ids = [i32(c["ids"]) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for s in range(2):
            outs[s].append(wq.wq_lora(xs[s], cases[s]["bank"], ids[s], ys[s], stream=streams[s]))
    torch.cuda.synchronize()
    for s in range(2):
        within(outs[s][0], cases[s]["want"], cases[s]["bound"])
        assert all(torch.equal(o, outs[s][0]) for o in outs[s])
