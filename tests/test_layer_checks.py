"""The norm's, rotary positions', adapters' and page tables' entry points refuse what they do not cover, before anything
is launched (CPU), and the references of their GPU tests agree with plain statements of the definitions."""
import ctypes
import math
import os

import pytest
import torch

import _layer
import weight_only_quantized_w4a16_amd as wq

P = ctypes.c_void_p
ends_of = lambda *e: (ctypes.c_int32 * len(e))(*e)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(wq.LIB_PATH):
        from weight_only_quantized_w4a16_amd import build
        build.build()
    return wq.lib()


# Fake, never-dereferenced pointers: validation must return before any launch.
def norm_call(L, x=1 << 20, ld_x=1024, r=None, ld_r=1024, w=256, eps=1e-5, dt=0, y=2 << 20, ld_y=1024, s=None,
              ld_s=1024, rows=4, heads=8, dim=128):
    return L.wq_rms_norm(P(x), ld_x, P(r), ld_r, P(w), eps, dt, P(y), ld_y, P(s), ld_s, rows, heads, dim, None)


def test_norm_refusals(L):
    assert norm_call(L, rows=0) == 0
    for eps in (0.0, -1e-5, 1e-40, float("inf"), float("nan")):
        assert norm_call(L, eps=eps) == 1
    assert norm_call(L, dt=2) == 1
    assert norm_call(L, rows=-1) == 1
    assert norm_call(L, heads=0) == 1
    assert norm_call(L, dim=0) == 1
    assert norm_call(L, dim=124) == 2
    assert norm_call(L, heads=1, dim=65544, ld_x=1 << 17, ld_y=1 << 17) == 2
    assert norm_call(L, heads=8192, dim=8, ld_x=1 << 16, ld_y=1 << 16) == 2
    assert norm_call(L, rows=1 << 24, heads=4096, dim=8, ld_x=1 << 16, ld_y=1 << 16) == 2
    assert norm_call(L, x=None) == 1
    assert norm_call(L, y=None) == 1
    assert norm_call(L, w=None) == 1
    assert norm_call(L, w=264) == 2
    assert norm_call(L, x=(1 << 20) + 8) == 2
    assert norm_call(L, ld_x=1028) == 2
    assert norm_call(L, ld_y=1016) == 1
    assert norm_call(L, s=3 << 20) == 1                       # a sum without a residual
    assert norm_call(L, y=(1 << 20) + 16) == 1                # over its input, elsewhere
    assert norm_call(L, y=1 << 20, ld_y=2048) == 1            # over its input with another stride
    assert norm_call(L, r=3 << 20, y=(3 << 20) + 2048) == 1
    assert norm_call(L, r=3 << 20, s=2 << 20) == 1            # both outputs in one place
    assert norm_call(L, r=3 << 20, s=(2 << 20) + 1024) == 1
    assert norm_call(L, w=(2 << 20) + 3 * 2048) == 1          # over the weight
    assert norm_call(L, r=3 << 20, s=4 << 20, w=4 << 20) == 1


def test_norm_overlaps_by_counting(L):
    """What shares elements is refused, what lies between the rows is not (the weight's alignment is looked at last)."""
    base, rows, width = 1 << 20, 3, 64
    for ld_x, ld_y in ((64, 64), (128, 128), (136, 136), (192, 128), (72, 200)):
        xe = {base + 2 * (i * ld_x + j) for i in range(rows) for j in range(width)}
        for d in range(-2 * 3 * 200, 2 * 3 * 200, 48):
            d = d // 16 * 16
            y = base + d
            meets = any(y + 2 * (i * ld_y + j) in xe for i in range(rows) for j in range(width))
            if y == base and ld_x == ld_y:
                meets = False
            got = norm_call(L, x=base, ld_x=ld_x, y=y, ld_y=ld_y, w=(4 << 20) + 8, rows=rows, heads=1, dim=width)
            assert got == (1 if meets else 2), (ld_x, ld_y, d)
            # a weight among the output's rows
            w = base + d
            meets = any(w + 2 * j in xe for j in range(width))
            got = norm_call(L, x=4 << 20, ld_x=64, y=base, ld_y=ld_x, w=w, rows=rows, heads=1, dim=width, r=5 << 20,
                            ld_r=64, s=6 << 20, ld_s=64) if meets else 1
            assert got == 1


def rotary_call(L, q=1 << 20, ld_q=1536, k=(1 << 20) + 2048, ld_k=1536, dt=0, turns=64, axis=None, factor=1.0, pos=None,
                ld_pos=0, lens=64, cu=None, qo=1 << 20, ld_qo=1536, ko=(1 << 20) + 2048, ld_ko=1536, rows=4, batch=2,
                q_heads=8, kv_heads=2, D=128, R=128, adjacent=0, axes=1):
    return L.wq_rotary(P(q), ld_q, P(k), ld_k, dt, P(turns), P(axis), factor, P(pos), ld_pos, P(lens), P(cu), P(qo), ld_qo,
                       P(ko), ld_ko, rows, batch, q_heads, kv_heads, D, R, adjacent, axes, None)


def test_rotary_refusals(L):
    assert rotary_call(L, rows=0, batch=0) == 0
    assert rotary_call(L, rows=0, pos=64) == 0
    assert rotary_call(L, dt=2) == 1
    assert rotary_call(L, R=130) == 1
    assert rotary_call(L, R=0) == 1
    assert rotary_call(L, R=31) == 1
    assert rotary_call(L, R=40) == 2                          # halves not 16-byte aligned
    assert rotary_call(L, R=36, adjacent=1) == 2
    assert rotary_call(L, D=132, ld_q=2112, ld_k=2112, ld_qo=2112, ld_ko=2112) == 2
    assert rotary_call(L, D=520, R=512, ld_q=8192, ld_k=8192, ld_qo=8192, ld_ko=8192) == 2
    assert rotary_call(L, adjacent=2) == 1
    assert rotary_call(L, axes=0) == 1
    assert rotary_call(L, axes=17) == 2
    assert rotary_call(L, factor=float("inf")) == 1
    assert rotary_call(L, factor=float("nan")) == 1
    assert rotary_call(L, rows=-1) == 1
    assert rotary_call(L, rows=3) == 1                        # 3 rows of 2 sequences without offsets
    assert rotary_call(L, batch=0) == 1
    assert rotary_call(L, lens=None) == 1
    assert rotary_call(L, rows=1 << 25, batch=1) == 2
    assert rotary_call(L, turns=None) == 1
    assert rotary_call(L, turns=68) == 2
    assert rotary_call(L, q=None) == 1
    assert rotary_call(L, qo=None) == 1
    assert rotary_call(L, k=None) == 1                        # keys announced and missing
    assert rotary_call(L, kv_heads=0) == 1                    # and the other way round
    assert rotary_call(L, ko=None) == 1
    assert rotary_call(L, q=(1 << 20) + 8) == 2
    assert rotary_call(L, ld_k=1540) == 2
    assert rotary_call(L, ld_qo=512) == 1
    assert rotary_call(L, pos=64, axes=3, ld_pos=3) == 1      # axes would share positions
    assert rotary_call(L, pos=64, ld_pos=-1) == 1
    assert rotary_call(L, qo=(1 << 20) + 256) == 1            # over other rows or heads of its input
    assert rotary_call(L, ko=1 << 20) == 1                    # keys over queries
    assert rotary_call(L, qo=2 << 20, ko=(2 << 20) + 16) == 1
    assert rotary_call(L, qo=(1 << 20) + 2048, ko=2 << 20) == 1


def lora_call(L, x=1 << 20, dt=0, a=2 << 20, b=3 << 20, scales=64, ranks=None, ids=64, cu=None, y=4 << 20, out=5 << 20,
              rows=100, batch=2, num=2, N=512, K=256, rank=16, slices=1, ends=ends_of(512), ws=6 << 20, ws_bytes=1 << 16):
    return L.wq_lora(P(x), dt, P(a), P(b), P(scales), P(ranks), P(ids), P(cu), P(y), P(out), rows, batch, num, N, K, rank,
                     slices, ends, P(ws), ws_bytes, None)


def test_lora_refusals(L):
    assert lora_call(L, rows=0, batch=0) == 0
    assert lora_call(L, dt=2) == 1
    assert lora_call(L, num=0) == 1
    assert lora_call(L, rank=0) == 1
    assert lora_call(L, rank=12) == 2
    assert lora_call(L, rank=136) == 2
    assert lora_call(L, K=192) == 2
    assert lora_call(L, N=520, ends=ends_of(520)) == 2
    assert lora_call(L, slices=2, ends=ends_of(256, 256)) == 1
    assert lora_call(L, slices=2, ends=ends_of(256, 496)) == 1
    assert lora_call(L, slices=2, ends=ends_of(248, 512)) == 2
    assert lora_call(L, slices=2, ends=ends_of(-16, 512)) == 1
    assert lora_call(L, slices=5, ends=ends_of(16, 32, 48, 64, 512)) == 2
    assert lora_call(L, ends=None) == 1
    assert lora_call(L, rows=-1) == 1
    assert lora_call(L, rows=3) == 1
    assert lora_call(L, batch=0) == 1
    assert lora_call(L, rows=1 << 25, batch=1) == 2
    assert lora_call(L, rows=1 << 24, batch=1, N=1 << 20, ends=ends_of(1 << 20)) == 2
    for name in ("x", "a", "b", "scales", "ids", "y", "out"):
        assert lora_call(L, **{name: None}) == 1, name
    for name in ("x", "a", "b", "y", "out"):
        assert lora_call(L, **{name: (8 << 20) + 8}) == 2, name
    assert lora_call(L, out=(4 << 20) + 1024) == 1            # over other rows of y
    assert lora_call(L, out=1 << 20) == 1                     # over x, a, b
    assert lora_call(L, out=2 << 20) == 1
    assert lora_call(L, out=3 << 20) == 1
    assert lora_call(L, ws=None) == 4
    assert lora_call(L, ws_bytes=8) == 4
    assert lora_call(L, ws=(6 << 20) + 8) == 2
    assert lora_call(L, ws=5 << 20) == 1                      # over out, a, b
    assert lora_call(L, ws=2 << 20) == 1
    assert lora_call(L, ws=3 << 20) == 1
    need = wq.wq_lora_workspace_bytes(100, 2, 256, 16)
    assert need >= 100 * 16 * 4 and lora_call(L, ws_bytes=need - 1) == 4
    # a few rows of a small adapter need none (an output that overlaps is looked at before)
    assert wq.wq_lora_workspace_bytes(4, 2, 256, 16) == 0
    assert lora_call(L, rows=4, ws=None, ws_bytes=0, out=1 << 20) == 1
    for bad in ((0, 1, 256, 16, 1), (4, 2, 200, 16, 1), (4, 2, 256, 20, 1), (4, 2, 256, 16, 5), (4, 0, 256, 16, 1)):
        assert wq.wq_lora_workspace_bytes(*bad) == 0, bad


def resize_call(L, table=1 << 20, lens=2 << 20, want=3 << 20, free=4 << 20, counts=5 << 20, cu=6 << 20, pos=7 << 20,
                slots=8 << 20, rows=16, batch=4, max_pages=8, num_pages=32, page=16, ws=9 << 20, ws_bytes=1 << 16):
    return L.wq_kv_resize(P(table), P(lens), P(want), P(free), P(counts), P(cu), P(pos), P(slots), rows, batch, max_pages,
                          num_pages, page, P(ws), ws_bytes, None)


def test_resize_refusals(L):
    assert resize_call(L, rows=-1) == 1
    assert resize_call(L, batch=-1) == 1
    assert resize_call(L, num_pages=0) == 1
    assert resize_call(L, page=24) == 2
    assert resize_call(L, page=8) == 2
    assert resize_call(L, page=2048) == 2
    assert resize_call(L, batch=1 << 17) == 2
    assert resize_call(L, rows=1 << 25) == 2
    assert resize_call(L, max_pages=1 << 27) == 2
    for name in ("table", "lens", "want", "free", "counts"):
        assert resize_call(L, **{name: None}) == 1, name
    assert resize_call(L, table=(1 << 20) + 2) == 2
    assert resize_call(L, slots=(8 << 20) + 4) == 2
    # (a small step needs no scratch; an output that overlaps is looked at behind it)
    assert wq.wq_kv_resize_workspace_bytes(4, 8, 32, 16) == 0
    assert resize_call(L, ws=None, ws_bytes=0, cu=2 << 20) == 1
    need = wq.wq_kv_resize_workspace_bytes(4, 8, 32, 1 << 14)
    assert need > 0
    assert resize_call(L, rows=1 << 14, ws=None, slots=16 << 20) == 4
    assert resize_call(L, rows=1 << 14, ws_bytes=need - 1, slots=16 << 20) == 4
    assert resize_call(L, rows=1 << 14, ws=(9 << 20) + 8, slots=16 << 20) == 2
    assert resize_call(L, want=2 << 20) == 1                  # lengths over wanted lengths
    assert resize_call(L, cu=(2 << 20) + 8) == 1
    assert resize_call(L, pos=(1 << 20) + 124) == 1           # over the table's last entry
    assert resize_call(L, slots=(7 << 20) + 56) == 1
    assert resize_call(L, counts=(4 << 20) + 124) == 1
    assert wq.wq_kv_resize_workspace_bytes(-1, 8, 32, 0) == 0
    assert wq.wq_kv_resize_workspace_bytes(1 << 17, 8, 32, 0) == 0


def test_ranges_meet_by_counting(L):
    """Overlaps of row matrices of different widths (queries over keys), against counting."""
    base = 1 << 20
    for ld_q, ld_k, rows in ((1536, 1536, 3), (1024, 256, 4), (1032, 1536, 2)):
        for d in list(range(-4096, 4097, 304)) + [-512, -2048, 2048, 512]:
            d = d // 16 * 16
            k = base + (1 << 12) + d
            qe = {base + (1 << 12) + 2 * (i * ld_q + j) for i in range(rows) for j in range(1024)}
            meets = any(k + 2 * (i * ld_k + j) in qe for i in range(rows) for j in range(256))
            got = rotary_call(L, q=base + (1 << 12), ld_q=ld_q, qo=base + (1 << 12), ld_qo=ld_q, k=4 << 20, ld_k=ld_k, ko=k,
                              ld_ko=ld_k, rows=rows, batch=1, turns=68, kv_heads=2)
            # (what is not refused for its overlap ends at the plan's misaligned pointer)
            assert got == (1 if meets else 2), (ld_q, ld_k, rows, d)


def test_plan_and_bank_and_pages_checks():
    plan = wq.wq_rotary_plan(128, device="cpu")
    assert plan.num_axes == 1 and plan.axis is None and plan.rotary_dim == 128
    # pair 0 turns by 1 radian, the others by base^(-2 i / 128)
    u = int(plan.turns[0]) % 2 ** 64
    assert abs(u / 2.0 ** 64 - 1 / (2 * math.pi)) < 1e-15
    three = wq.wq_rotary_plan(128, sections=(16, 24, 24), device="cpu")
    assert three.num_axes == 3 and three.axis.tolist() == [0] * 16 + [1] * 24 + [2] * 24
    assert wq.wq_rotary_plan(64, axes=[0, 1] * 16, device="cpu").num_axes == 2
    assert wq.wq_rotary_plan(64, axes=[0] * 32, device="cpu").num_axes == 1
    assert (wq.wq_rotary_plan(64, freqs=[-1.0] * 32, device="cpu").turns + wq.wq_rotary_plan(
        64, freqs=[1.0] * 32, device="cpu").turns).abs().max() <= 1 << 12
    for bad in (dict(freqs=[1.0]), dict(freqs=[math.inf] * 32), dict(sections=(16, 17)), dict(axes=[0]), dict(base=0.0),
                dict(sections=(32,), axes=[0] * 32), dict(axes=[-1] * 32), dict(rotary_dim=80), dict(factor=math.nan)):
        with pytest.raises(ValueError):
            wq.wq_rotary_plan(64, device="cpu", **bad)
    h = dict(dtype=torch.float16)
    a, b, s = torch.zeros(2, 3, 16, 256, **h), torch.zeros(2, 512, 16, **h), torch.ones(2)
    bank = wq.LoraBank(a, b, s, slices=(256, 128, 128))
    assert (bank.count, bank.rank, bank.K, bank.N, bank.num_slices, list(bank.ends)) == (2, 16, 256, 512, 3, [256, 384, 512])
    assert wq.LoraBank(a[:, 0].contiguous(), b, s).num_slices == 1
    for bad in (dict(slices=(256, 256)), dict(slices=None), dict(slices=(256, 0, 256)), dict(b=b[:1]), dict(b=b.float()),
                dict(scales=s.double()), dict(ranks=torch.ones(2)), dict(a=a.transpose(2, 3)), dict(a=a.float())):
        with pytest.raises(ValueError):
            wq.LoraBank(**{**dict(a=a, b=b, scales=s, slices=(256, 128, 128)), **bad})
    pages = wq.wq_kv_pages(8, 16, 2, 4, device="cpu")
    assert pages.free.tolist() == list(range(7, -1, -1)) and pages.counts.tolist() == [8, 0]
    assert pages.block_table.eq(-1).all() and pages.kv_lens.tolist() == [0, 0]
    for bad in (dict(page_size=24), dict(num_pages=9), dict(kv_lens=torch.zeros(3, dtype=torch.int32)),
                dict(counts=torch.zeros(2))):
        with pytest.raises(ValueError):
            wq.KVPages(**{**dict(block_table=pages.block_table, kv_lens=pages.kv_lens, free=pages.free, counts=pages.counts,
                                 num_pages=8, page_size=16), **bad})


def test_binding_refuses_before_the_library(L):
    """Wrong shapes, types and devices become Python errors (CPU tensors: the last check is for the GPU)."""
    x, w = torch.zeros(4, 64).half(), torch.ones(64).half()

    def refused(f, *a, **k):
        with pytest.raises(ValueError) as e:
            f(*a, **k)
        return str(e.value)

    assert "GPU" in refused(wq.wq_rms_norm, x, w)
    assert "GPU" in refused(wq.wq_rms_norm, x, w, residual=x, out=x, sum_out=x.clone())
    assert "weight" in refused(wq.wq_rms_norm, x, w[:32])
    assert "weight" in refused(wq.wq_rms_norm, x, w.float())
    assert "dtype" in refused(wq.wq_rms_norm, x.float(), w)
    assert "residual" in refused(wq.wq_rms_norm, x, w, residual=x[:3])
    assert "residual" in refused(wq.wq_rms_norm, x, w, sum_out=x)
    assert "eps" in refused(wq.wq_rms_norm, x, w, 0.0)
    assert "out" in refused(wq.wq_rms_norm, x, w, out=x[:, :32])
    assert "contiguous" in refused(wq.wq_rms_norm, torch.zeros(64, 4).half().t(), w)
    assert "stride" in refused(wq.wq_rms_norm, torch.zeros(4, 68).half()[:, :64], w)
    plan = wq.wq_rotary_plan(64, device="cpu")
    q, k = torch.zeros(4, 8, 64).half(), torch.zeros(4, 2, 64).half()
    lens = torch.tensor([2, 3], dtype=torch.int32)
    assert "GPU" in refused(wq.wq_rotary, q, k, plan, kv_lens=lens)
    assert "GPU" in refused(wq.wq_rotary, q, None, plan, positions=torch.zeros(4, dtype=torch.int32))
    assert "kv_lens" in refused(wq.wq_rotary, q, k, plan)
    assert "either" in refused(wq.wq_rotary, q, k, plan, positions=torch.zeros(4, dtype=torch.int32), kv_lens=lens)
    assert "positions" in refused(wq.wq_rotary, q, k, plan, positions=torch.zeros(4))
    assert "positions" in refused(wq.wq_rotary, q, k, plan, positions=[0, 1, 2, 3])
    assert "positions" in refused(wq.wq_rotary, q, k, plan, positions=torch.zeros(2, 4, dtype=torch.int32))
    assert "k must" in refused(wq.wq_rotary, q, k[:3], plan, kv_lens=lens)
    assert "channels" in refused(wq.wq_rotary, torch.zeros(4, 8, 32).half(), k, plan, kv_lens=lens)
    assert "out[1]" in refused(wq.wq_rotary, q, None, plan, kv_lens=lens, out=(q, k))
    assert "rows" in refused(wq.wq_rotary, q[:3], k[:3], plan, kv_lens=lens)
    bank = wq.LoraBank(torch.zeros(2, 16, 256).half(), torch.zeros(2, 64, 16).half(), torch.ones(2))
    x, y, ids = torch.zeros(100, 256).half(), torch.zeros(100, 64).half(), torch.zeros(2, dtype=torch.int32)
    assert "GPU" in refused(wq.wq_lora, x, bank, ids, y)
    assert "K" in refused(wq.wq_lora, x[:, :128], bank, ids, y)
    assert "bank" in refused(wq.wq_lora, x.bfloat16(), bank, ids, y.bfloat16())
    assert "y must" in refused(wq.wq_lora, x, bank, ids, y[:3])
    assert "adapters" in refused(wq.wq_lora, x, bank, ids.long(), y)
    assert "cu_q" in refused(wq.wq_lora, x, bank, ids, y, cu_q=ids)
    assert "sequence" in refused(wq.wq_lora, x, bank, torch.zeros(3, dtype=torch.int32), y)
    assert "ws" in refused(wq.wq_lora, x, bank, ids, y, ws=torch.zeros(1))
    pages = wq.wq_kv_pages(8, 16, 2, 4, device="cpu")
    assert "GPU" in refused(wq.wq_kv_resize, pages, lens)
    assert "want_lens" in refused(wq.wq_kv_resize, pages, lens.long())
    assert "rows" in refused(wq.wq_kv_resize, pages, lens, -1)
    assert "slots" in refused(wq.wq_kv_resize, pages, lens, 4, slots=torch.zeros(4, dtype=torch.int32))


def test_references():
    """The references against plain statements of the definitions."""
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(3, 40, generator=g).half(), torch.randn(40, generator=g).half()
    y = _layer.rms_norm(x, w, 1e-5)[0]
    for t in range(3):
        ms = math.fsum(float(v) ** 2 for v in x[t]) / 40
        for c in range(40):
            assert math.isclose(float(y[t, c]), float(w[c]) * float(x[t, c]) / math.sqrt(ms + 1e-5), rel_tol=1e-12)
    x = torch.randn(2, 1, 12, generator=g).half()
    pos, freqs, axis = torch.tensor([[5, 1000003], [7, 2]]), [1.0, 0.37, 1e-3, 2.5], [0, 1, 1, 0]
    for adjacent in (False, True):
        out = _layer.rotary(x, pos, freqs, axis, adjacent, 1.5)[0]
        for t in range(2):
            for i in range(4):
                m, n = (2 * i, 2 * i + 1) if adjacent else (i, i + 4)
                z = complex(x[t, 0, m], x[t, 0, n]) * 1.5 * complex(math.cos(float(pos[axis[i], t]) * freqs[i]),
                                                                   math.sin(float(pos[axis[i], t]) * freqs[i]))
                assert abs(complex(out[t, 0, m], out[t, 0, n]) - z) < 1e-12
            assert torch.equal(out[t, 0, 8:], x[t, 0, 8:].double())
    x, y = torch.randn(2, 6, generator=g).half(), torch.randn(2, 5, generator=g).half()
    a, b = torch.randn(2, 2, 3, 6, generator=g).half(), torch.randn(2, 5, 3, generator=g).half()
    out = _layer.lora(x, y, a, b, [0.5, 2.0], [3, 2], (2, 3), [1, -1])[0]
    for n in range(5):
        s = 0 if n < 2 else 1
        want = float(y[0, n]) + 2.0 * sum(float(b[1, n, j]) * sum(float(a[1, s, j, k]) * float(x[0, k]) for k in range(6))
                                          for j in range(2))
        assert math.isclose(float(out[0, n]), want, rel_tol=1e-12, abs_tol=1e-12)
    assert torch.equal(out[1], y[1].double())
    p = _layer.Pages([[4, 5, -1], [6, -1, -1]], [20, 3], [0, 1, 2, 3, 9, 9, 9], 4, 16)
    before = ([list(r) for r in p.table], list(p.free), p.count)
    cu, pos, slots = p.resize([40, 20], 38)
    assert cu == [0, 20, 37] and pos == list(range(20, 40)) + list(range(3, 20)) + [-1]
    assert p.table == [[4, 5, 3], [6, 2, -1]] and p.count == 2 and slots[0] == 5 * 16 + 4 and slots[12] == 48
    p.resize([20, 3], 0)
    assert (p.table, p.free, p.count) == before
    p.resize([0, 48], 0)  # one ends, the other takes its pages
    assert p.table == [[-1, -1, -1], [6, 4, 5]] and p.count == 4
    assert p.resize([20, 49], 1) == ([0, 0, 0], [-1], [-1]) and p.lack == -1
    assert p.resize([48, 48], 1)[0] == [0, 48, 48] and p.count == 1
    p = _layer.Pages([[-1] * 3], [0], [7, 8], 2, 16)
    assert p.resize([48], 0) == ([0, 0], [], []) and p.lack == 1 and p.lens == [0]
