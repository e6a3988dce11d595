"""Whole decoder layers: page tables, norms, adapters and rotary positions with the products, the cache and attention
(weight_only_quantized_w4a16_amd.stack.CachedStack).

Every part is checked on the very input the GPU used, against the oracle or a 64-bit reference; sequences come, grow
and end between the steps; a step captured with its page tables is replayed as they do."""
import numpy as np
import pytest
import torch

import _kv
import _layer
import workloads as wl
from _util import bits_to_tensor, oracle_y, repack_layer, tensor_bits, tensor_f64, within_tolerance
from test_gpu_gate_up import gate_up_bound, repack_gate_up

pytestmark = pytest.mark.gpu
DIM, INTER, H, KV, D = 512, 768, 8, 2, 64
QKV = (H + 2 * KV) * D
SLICES = (H * D, KV * D, KV * D)
RANK, ADAPTERS, EPS = 16, 4, 1e-5
RANKS = [16, 5, 8, 16]


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.fixture(scope="module")
def wq():
    import weight_only_quantized_w4a16_amd as m
    m.lib()
    assert torch.cuda.is_available()
    return m


@pytest.fixture(scope="module")
def model(wq):
    from weight_only_quantized_w4a16_amd.stack import DecoderWeights, LayerAdapters
    g = torch.Generator().manual_seed(11)
    layers, raw, banks, norms, bias = [], [], [], [], []
    for li in range(2):
        Ls = {}
        for j, (name, K, N) in enumerate((("qkv", DIM, QKV), ("o", H * D, DIM), ("gate_up", DIM, 2 * INTER),
                                          ("down", INTER, DIM))):
            c = 0.5 / np.sqrt(13.0 / 12.0 * 22.6 * K)
            Ls[name] = wl.make_layer(K, N, 4, 128, wl.ZERO_F16, 300 * li + j, scale_range=(0.5 * c, 1.5 * c),
                                     zero_range=(5.5, 9.5))
        layers.append(DecoderWeights(repack_layer(wq, Ls["qkv"]), repack_layer(wq, Ls["o"]),
                                     repack_gate_up(wq, Ls["gate_up"]), repack_layer(wq, Ls["down"])))
        raw.append(Ls)
        bank = {}
        for name, K, slices in (("qkv", DIM, SLICES), ("o", H * D, (DIM,)), ("down", INTER, (DIM,))):
            a = (torch.randn(ADAPTERS, len(slices), RANK, K, generator=g) / K ** 0.5).half()
            b = (torch.randn(ADAPTERS, sum(slices), RANK, generator=g) * 0.3).half()
            bank[name] = wq.LoraBank(a.cuda(), b.cuda(), torch.tensor([0.5, 1.0, 2.0, -0.5]).cuda(), i32(RANKS), slices)
        banks.append(LayerAdapters(**bank))
        norms.append(tuple((1 + 0.2 * torch.randn(DIM, generator=g)).half().cuda() for _ in range(2)))
        bias.append((torch.randn(QKV, generator=g) * 0.3).half().cuda())
    return layers, raw, banks, norms, bias


def make_stack(wq, model, max_rows, rotary, pages=60):
    from weight_only_quantized_w4a16_amd.stack import CachedStack
    layers, _, banks, norms, bias = model
    return CachedStack(layers, H, KV, D, pages, max_rows, torch.float16, "cuda", qkv_bias=bias, norms=norms, eps=EPS,
                       rotary=rotary, adapters=banks)


def within(got, want, bound, what):
    assert bool(((got.cpu().double() - want).abs() <= bound).all()), what


def adapted_ok(orc, x, L, plus, bank, slices, ids, y, what):
    """y = x W + plus + the adapters' part: the product's tolerance, one more rounding (its own result's) and the
    adapters' bound."""
    ref = oracle_y(orc, tensor_bits(x), wl.F16, L)
    _, _, bound = within_tolerance(ref, ref)
    base = torch.from_numpy(ref + plus)
    want, err = _layer.lora(x.cpu(), base, bank.a.cpu(), bank.b.cpu(), bank.scales.cpu(), RANKS, slices, ids)
    want0 = base.abs().max()
    within(y, want, err + _layer.rounding(want, torch.float16) + bound + 2.0 ** -11 * float(want0) * 2, what)


def check(orc, rec, model, freqs, axis, hist, new, lens, ids, positions):
    layers, raw, banks, norms, bias = model
    row_ids = [i for i, n in zip(ids, new) for _ in range(n)]
    for r, Ls, A, (w1, w2), b in zip(rec, raw, banks, norms, bias):
        T = r["x"].shape[0]
        y, yb, _, _ = _layer.rms_norm(r["x"].cpu(), w1.cpu(), EPS)
        within(r["n1"], y, yb, "n1")
        adapted_ok(orc, r["n1"], Ls["qkv"], tensor_f64(b), A.qkv, SLICES, row_ids, r["unturned"], "qkv")
        before, heads = (r[n].view(T, H + 2 * KV, D).cpu() for n in ("unturned", "qkv"))
        want, bound = _layer.rotary(before[:, :H + KV], positions, freqs, axis, False, 1.0)
        within(heads[:, :H + KV], want, bound, "rotary")
        assert torch.equal(heads[:, H + KV:], before[:, H + KV:])
        at = 0
        for s, n in enumerate(new):
            rows = heads[at:at + n]
            K, V = hist[r["layer"]][s]
            K, V = torch.cat([K[:lens[s] - n], rows[:, H:H + KV]]), torch.cat([V[:lens[s] - n], rows[:, H + KV:]])
            hist[r["layer"]][s] = (K, V)
            if n:
                want, bound = _kv.attention(rows[:, :H], K, V, torch.arange(lens[s] - n, lens[s]), D ** -0.5, True, 0, D)
                within(r["attn"][at:at + n], want, bound, "attention")
            at += n
        adapted_ok(orc, r["attn"].reshape(T, H * D), Ls["o"], tensor_f64(r["x"]), A.o, (DIM,), row_ids, r["mid"], "o")
        y, yb, _, _ = _layer.rms_norm(r["mid"].cpu(), w2.cpu(), EPS)
        within(r["n2"], y, yb, "n2")
        L, nb = Ls["gate_up"], tensor_bits(r["n2"])
        h_ref = orc.linear_gate_up(nb, wl.F16, L.qweight, L.scales, L.zeros, L.mode, L.lut, L.g_idx, T, L.N, L.K, L.bits,
                                   L.group_size)
        assert np.all(np.abs(tensor_f64(r["h"]) - h_ref) <= gate_up_bound(oracle_y(orc, nb, wl.F16, L), h_ref, wl.F16))
        adapted_ok(orc, r["h"], Ls["down"], tensor_f64(r["mid"]), A.down, (DIM,), row_ids, r["y"], "down")


@pytest.mark.parametrize("axes", [1, 3])
def test_sequences_come_grow_and_end(orc, wq, model, axes):
    """Prompts, chunks, single tokens, a sequence cut back, one that ends and one in its place: every part of every
    step, with the pages that wq_kv_resize gave."""
    half = D // 2
    axis = [i * axes // half for i in range(half)]
    plan = wq.wq_rotary_plan(D, axes=axis if axes > 1 else None)
    freqs = [10000.0 ** (-i / half) for i in range(half)]
    st = make_stack(wq, model, 100, plan)
    pages = st.pages(4, 8)
    e = torch.empty(0, KV, D, dtype=torch.float16)
    hist = [[(e, e) for _ in range(4)] for _ in range(2)]
    g = torch.Generator().manual_seed(21)
    lens, ids = [0] * 4, [0, -1, 2, 3]
    for want in ([45, 3, 0, 20], [46, 23, 33, 20], [47, 24, 34, 21], [40, 24, 0, 21], [41, 25, 17, 22], [42, 26, 18, 23]):
        new = [max(0, b - a) for a, b in zip(lens, want)]
        lens = want
        T = sum(new)
        cu, pos, slots = wq.wq_kv_resize(pages, i32(want), T)
        assert pages.counts.tolist()[1] == 0 and cu.tolist() == [0] + list(np.cumsum(new))
        if T == 0:
            continue
        if want[2] == 17:
            ids[2] = 1
        x = torch.randn(T, DIM, generator=g).half().cuda()
        rec = []
        if axes == 1:
            y = st.step(x, pages.block_table, pages.kv_lens, cu, max_kv_len=64, record=rec, adapters=i32(ids))
            positions = pos[None].cpu()
        else:  # rows of an image: positions of their own
            positions = torch.stack([pos.cpu(), torch.randint(0, 40, (T,), generator=g), torch.randint(0, 40, (T,), generator=g)])
            positions = positions.to(torch.int32)
            y = st.step(x, pages.block_table, pages.kv_lens, cu, max_kv_len=64, record=rec, adapters=i32(ids),
                        positions=positions.cuda())
        assert torch.equal(rec[-1]["y"], y) and torch.equal(rec[1]["x"], rec[0]["y"])
        check(orc, rec, model, freqs, axis, hist, new, lens, ids, positions)


def test_a_step_with_its_pages_in_a_graph(wq, model):
    """Page tables, offsets and every layer in one graph: each replay takes the lengths and adapters it is given, a
    sequence that ends and one that begins among them, as the eager step does."""
    plan = wq.wq_rotary_plan(D)
    eager, st = make_stack(wq, model, 60, plan, 20), make_stack(wq, model, 60, plan, 20)
    g = torch.Generator().manual_seed(31)
    want, ids = i32([10, 20, 15]), i32([0, 1, -1])
    pe, pg = eager.pages(3, 6), st.pages(3, 6)
    x = torch.zeros(45, DIM, dtype=torch.float16, device="cuda")

    def step(stack, pages, rows):
        cu, _, _ = wq.wq_kv_resize(pages, want, rows)
        return cu, stack.step(x[:rows], pages.block_table, pages.kv_lens, cu, max_kv_len=96, adapters=ids)

    x.copy_(torch.randn(45, DIM, generator=g))
    a, b = step(eager, pe, 45)[1].clone(), step(st, pg, 45)[1].clone()
    assert torch.equal(a, b)
    want.copy_(i32([11, 21, 16]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cu, out = step(st, pg, 3)
    for lens, who in (([11, 21, 16], [0, 1, -1]), ([12, 22, 17], [0, 1, -1]), ([13, 0, 18], [2, 1, 3]), ([14, 1, 19], [2, 0, 3]),
                      ([33 * 96, 2, 20], [2, 0, 3]), ([15, 2, 20], [2, 0, 3])):
        want.copy_(i32(lens))
        ids.copy_(i32(who))
        x.copy_(torch.randn(45, DIM, generator=g))
        rows = step(eager, pe, 3)
        n = int(rows[0][-1])
        kept = rows[1][:n].clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cu, rows[0]) and torch.equal(out[:n], kept), lens
        for name in ("block_table", "kv_lens", "free", "counts"):
            assert torch.equal(getattr(pe, name), getattr(pg, name)), (name, lens)
    assert pg.kv_lens.tolist() == [15, 2, 20]


def test_refusals(wq, model):
    from weight_only_quantized_w4a16_amd.stack import CachedStack, LayerAdapters
    layers, _, banks, norms, bias = model
    args = (layers, H, KV, D, 8, 4, torch.float16, "cuda")
    with pytest.raises(ValueError, match="norm"):
        CachedStack(*args, norms=norms[:1])
    with pytest.raises(ValueError, match="rotary"):
        CachedStack(*args, rotary=wq.wq_rotary_plan(128))
    with pytest.raises(ValueError, match="per layer"):
        CachedStack(*args, adapters=banks[:1])
    with pytest.raises(ValueError, match="other products"):
        CachedStack(*args, adapters=[LayerAdapters(qkv=banks[0].o)] * 2)
    x = torch.zeros(1, DIM, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="adapter"):
        CachedStack(*args, adapters=banks).step(x, i32([[0]]), i32([1]))
    with pytest.raises(ValueError, match="adapter"):
        CachedStack(*args).step(x, i32([[0]]), i32([1]), adapters=i32([0]))
    with pytest.raises(ValueError, match="2 sequences need as many adapters"):
        CachedStack(*args, adapters=banks).step(x.repeat(2, 1), i32([[0], [1]]), i32([1, 1]), adapters=i32([0]))
    with pytest.raises(ValueError, match="positions"):
        CachedStack(*args).step(x, i32([[0]]), i32([1]), positions=i32([0]))
    # a product without adapters among those that have them
    some = [LayerAdapters(o=banks[0].o), LayerAdapters()]
    CachedStack(*args, adapters=some).step(x, i32([[0]]), i32([1]), adapters=i32([0]))
