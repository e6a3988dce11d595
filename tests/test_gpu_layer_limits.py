"""Page tables, adapters and rotary positions on the GPU where their numbers are largest or are none."""
import math

import pytest
import torch

import _layer
import weight_only_quantized_w4a16_amd as wq
from test_gpu_layer_ops import i32, randn, within

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    wq.lib()
    assert torch.cuda.is_available()


# ---------------------------------------------------------------------------- page tables
# (rows of the call, sequences): one workgroup, two launches, three launches
FORMS = [(0, 3), (5000, 3), (0, 1100)]


@pytest.mark.parametrize("rows,batch", FORMS)
@pytest.mark.parametrize("new", [(1 << 24) - 1, 1 << 24, (1 << 24) + 1, 20000003])
def test_resize_of_more_new_tokens_than_a_call_has_rows(rows, batch, new):
    """What a call numbers (rows <= 2^24) bounds its outputs, not what its sequences may grow by."""
    P, old = 1024, 5
    need = -(-(old + new) // P)
    pages = wq.wq_kv_pages(need + 9, P, batch, need + 2)
    wq.wq_kv_resize(pages, i32([0, old] + [0] * (batch - 2)))
    lens = [0, old + new] + [0] * (batch - 2)
    cu, pos, slots = wq.wq_kv_resize(pages, i32(lens), rows)
    assert pages.counts.tolist() == [9, 0] and pages.kv_lens.tolist() == lens
    assert cu.tolist() == [0, 0] + [new] * (batch - 1)
    # (pages are taken from 0 on)
    table = torch.full((batch, need + 2), -1, dtype=torch.int32)
    table[1, :need] = torch.arange(need, dtype=torch.int32)
    assert torch.equal(pages.block_table.cpu(), table)
    assert torch.equal(pos.cpu(), old + torch.arange(rows, dtype=torch.int32))
    assert torch.equal(slots.cpu(), old + torch.arange(rows))
    wq.wq_kv_resize(pages, i32([0] * batch))
    assert pages.counts.tolist() == [need + 9, 0] and bool((pages.block_table == -1).all())
    assert torch.equal(pages.free, torch.arange(need + 8, -1, -1, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("rows,batch,each", [(0, 2, 1 << 30), (5000, 2, 1 << 30), (0, 1100, 1 << 25)])
def test_resize_counts_new_tokens_in_31_bits(rows, batch, each):
    """2^31 new tokens of all sequences together are no change, one fewer are."""
    P, n = 1024, (1 << 31) // each
    total = (1 << 31) // P
    pages = wq.wq_kv_pages(total, P, batch, each // P)
    full = [each] * n + [0] * (batch - n)
    cu, pos, slots = wq.wq_kv_resize(pages, i32(full), rows)
    assert pages.counts.tolist() == [total, -1] and not cu.any() and not pages.kv_lens.any()
    assert bool((pages.block_table == -1).all()) and bool((pos == -1).all()) and bool((slots == -1).all())
    lens = [each - 1] + full[1:]
    cu, pos, slots = wq.wq_kv_resize(pages, i32(lens), rows)
    assert pages.counts.tolist() == [0, 0] and pages.kv_lens.tolist() == lens
    assert cu.tolist() == [min(each * b, 1 << 31) - (b > 0) for b in range(batch + 1)]
    assert torch.equal(pages.block_table[:n].cpu().flatten(), torch.arange(total, dtype=torch.int32))
    assert torch.equal(pos.cpu(), torch.arange(rows, dtype=torch.int32))
    assert torch.equal(slots.cpu(), torch.arange(rows))


# ---------------------------------------------------------------------------- adapters
@pytest.mark.parametrize("rows,rank", [(1, 16), (4, 8), (14, 16), (100, 16), (120, 64), (900, 32), (1300, 16), (1300, 128)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_an_infinite_weight_of_an_adapter(rows, rank, dtype):
    """One entry of A is infinite, and so is the first of x A^T: every column is the infinity that B makes of it, though
    the others are past fp16's range (as fp16 numbers they would be infinities of either sign).  The other adapter's
    rows hold."""
    g = torch.Generator().manual_seed(rows + rank)
    K, N = 256, 144
    x, y = (randn(g, rows, K) * 3000).to(dtype), randn(g, rows, N).to(dtype)
    x[:, 3] = torch.where(x[:, 3] < 0, -1.0, 1.0).to(dtype)
    a, b = (randn(g, 2, 1, rank, K) * 2).to(dtype), randn(g, 2, N, rank).to(dtype)
    b[:, :, 0] = torch.where(b[:, :, 0] < 0, -1.0, 1.0).to(dtype)
    scales = torch.tensor([2.0 ** -9, 2.0 ** -9])
    v = x.double() @ a[0, 0, 1:].double().t().contiguous()
    assert rank < 16 or bool((v.abs().amax(1) > 65504).all())
    a[0, 0, 0, 3] = math.inf
    cut = rows if rows == 1 else rows // 2 + 1
    cu, ids = [0, cut, rows], [0, 1]
    bank = wq.LoraBank(a.cuda(), b.cuda(), scales.cuda())
    got = wq.wq_lora(x.cuda(), bank, i32(ids), y.cuda(), cu_q=i32(cu)).cpu()
    sign = x[:cut, 3].double()[:, None] * b[0, :, 0].double()[None]
    assert torch.equal(got[:cut].double(), sign * math.inf)
    if cut < rows:
        want, bound = _layer.lora(x[cut:], y[cut:], a, b, scales, [rank, rank], (N,), [1] * (rows - cut))
        within(got[cut:], want, bound)


# ---------------------------------------------------------------------------- numbers that are none
def guarded(shape, dtype, fill):
    """A tensor of `shape` in the middle of a larger buffer, all of it `fill`; and a check that the rest still is."""
    n, guard = math.prod(shape), 1 << 16
    whole = torch.full((n + 2 * guard,), fill, dtype=dtype, device="cuda")
    return whole[guard:guard + n].view(shape), lambda: bool((whole[:guard] == fill).all() and (whole[guard + n:] == fill).all())


ODD = [lambda n, T: [0] * (n + 1), lambda n, T: [1 << 30] * (n + 1), lambda n, T: [-2147483648] * (n + 1),
       lambda n, T: [(-5, 3, 2, 9, 4, 1 << 30, 3)[i % 7] for i in range(n + 1)],
       lambda n, T: [T - 7 * i for i in range(n + 1)], lambda n, T: [2147483647] * n + [-1]]


@pytest.mark.parametrize("rows,batch,rank", [(12, 6, 16), (70, 6, 16), (70, 90, 24), (1300, 6, 16), (1300, 90, 64), (700, 700, 8)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_offsets_that_are_none_stay_within_the_buffers(rows, batch, rank, dtype):
    """Nothing but the outputs and the scratch is written, whatever the offsets say; where they give no sequence a row,
    no row is."""
    g = torch.Generator().manual_seed(rows + batch)
    K, N = 256, 80
    x, y = randn(g, rows, K).to(dtype).cuda(), randn(g, rows, N).to(dtype).cuda()
    bank = wq.LoraBank(randn(g, 4, 1, rank, K).to(dtype).cuda(), randn(g, 4, N, rank).to(dtype).cuda(),
                       torch.ones(4, device="cuda"))
    ids, lens = i32([b % 6 - 1 for b in range(batch)]), i32([b % 9 for b in range(batch)])
    plan, q, k = wq.wq_rotary_plan(64), randn(g, rows, 3, 64).to(dtype).cuda(), randn(g, rows, 1, 64).to(dtype).cuda()
    need = wq.wq_lora_workspace_bytes(rows, batch, K, rank)
    for i, odd in enumerate(ODD):
        cu = i32(odd(batch, rows))
        out, out_kept = guarded((rows, N), dtype, 7.0)
        ws, ws_kept = guarded((max(need, 16),), torch.uint8, 0xFF)
        wq.wq_lora(x, bank, ids, y, cu_q=cu, out=out, ws=ws)
        qo, q_kept = guarded((rows, 3, 64), dtype, 7.0)
        ko, k_kept = guarded((rows, 1, 64), dtype, 7.0)
        wq.wq_rotary(q, k, plan, kv_lens=lens, cu_q=cu, out=(qo, ko))
        assert out_kept() and ws_kept() and q_kept() and k_kept(), i
        if i < 3:
            assert bool((out == 7).all()) and bool((qo == 7).all()) and bool((ko == 7).all()), i


@pytest.mark.parametrize("rows,batch", [(40, 5), (6000, 5), (40, 1100)])
def test_page_tables_that_are_none_stay_within_the_buffers(rows, batch):
    """Lengths, counts and entries of the tables that make no sense: nothing but the tables and the outputs is written,
    and the verdict is what the rules make of them."""
    g = torch.Generator().manual_seed(rows + batch)
    P, max_pages, num_pages = 16, 30, 400
    pages_of = lambda n: -(-n // P)
    some = torch.tensor([0, 1, 17, 400, 480, 481, -1, 1 << 30, 2147483647, -2147483648])
    pick = lambda *shape: some[torch.randint(0, len(some), shape, generator=g)].to(torch.int32).cuda()
    for step in range(20):
        checks, t = [], {}
        for name, shape, values in (("block_table", (batch, max_pages), pick(batch, max_pages)), ("kv_lens", (batch,), pick(batch)),
                                    ("free", (num_pages,), pick(num_pages)), ("counts", (2,), pick(2))):
            t[name], kept = guarded(shape, torch.int32, 7)
            t[name].copy_(values)
            checks.append(kept)
        if step % 2:  # (not all of it at once: some of these are changes)
            t["kv_lens"].copy_(torch.randint(0, 40, (batch,), generator=g))
            t["counts"][0] = [0, 33, num_pages][step % 3]
        if step % 4 == 3:
            t["kv_lens"][5:] = 0
        want = pick(batch)
        if step % 4 > 1:
            few = torch.rand(batch, generator=g) < 60 / batch
            want = torch.where(few, torch.randint(0, 90, (batch,), generator=g), 0).to(torch.int32).cuda()
        pages = wq.KVPages(**t, num_pages=num_pages, page_size=P)
        outs = []
        for n, dtype in ((batch + 1, torch.int32), (rows, torch.int32), (rows, torch.int64)):
            o, kept = guarded((n,), dtype, 7)
            outs.append(o)
            checks.append(kept)
        before = {name: v.clone() for name, v in t.items()}
        wq.wq_kv_resize(pages, want, rows, *outs)
        assert all(kept() for kept in checks), step
        old, new = (before["kv_lens"].long().clamp(0, max_pages * P).tolist(), want.tolist())
        moved = [pages_of(m) - pages_of(n) for n, m in zip(old, new)]
        top = min(max(int(before["counts"][0]), 0), num_pages) - sum(d for d in moved if d < 0)
        fails = any(not 0 <= m <= max_pages * P for m in new) or top > num_pages
        status = -1 if fails else max(0, sum(d for d in moved if d > 0) - top)
        assert int(t["counts"][1]) == status, step
        if status:
            assert all(torch.equal(t[n], before[n]) for n in ("block_table", "kv_lens", "free")) and not outs[0].any()
        else:
            assert torch.equal(t["kv_lens"], want) and outs[0].tolist() == [
                sum(max(0, m - n) for n, m in zip(old[:b], new[:b])) for b in range(batch + 1)]
