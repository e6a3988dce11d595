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
