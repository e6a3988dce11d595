"""The 4-bit key/value cache's entry points refuse what they do not cover, before anything is launched (CPU), and
the reference of its GPU tests agrees with a plain statement of the definition."""
import ctypes
import fractions
import os

import pytest
import torch

import _kv
import weight_only_quantized_w4a16_amd as wq

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(wq.LIB_PATH):
        from weight_only_quantized_w4a16_amd import build
        build.build()
    return wq.lib()


def test_cache_bytes(L):
    # 16 tokens of one head: 16 D bytes of codes, 128 bytes of steps and offsets per group
    assert wq.wq_kv_cache_bytes(10, 64, 8, 128, 128) == 10 * 4 * 8 * (16 * 128 + 128)
    assert wq.wq_kv_cache_bytes(1, 16, 1, 256, 32) == 16 * 256 + 8 * 128
    assert wq.wq_kv_cache_bytes(1 << 20, 16, 8, 64, 64) == (1 << 20) * 8 * 1152  # past 32 bits
    for bad in ((0, 16, 1, 64, 64), (1, 8, 1, 64, 64), (1, 48, 1, 64, 64), (1, 2048, 1, 64, 64), (1, 16, 0, 64, 64),
                (1, 16, 1, 80, 16), (1, 16, 1, 64, 128), (1, 16, 1, 96, 64), (1, 16, 1, 128, 16), (1, 16, 1, 512, 128),
                (1 << 28, 1024, 8, 64, 64), (-1, 16, 1, 64, 64)):
        assert wq.wq_kv_cache_bytes(*bad) == 0, bad


def rows_call(L, fn, k=128, v=128, ld_k=512, ld_v=512, dt=0, cache=128, table=4, lens=4, cu=None, rows=2, batch=2,
              max_pages=1, num_pages=4, page=16, heads=4, D=128, G=128):
    # fake, never-dereferenced pointers: validation must return before any launch
    a = [P(k), P(v), ld_k, ld_v, dt, P(cache)] if fn == "wq_kv_write" else [P(cache), P(k), P(v), ld_k, ld_v, dt]
    return getattr(L, fn)(*a, P(table), P(lens), P(cu), rows, batch, max_pages, num_pages, page, heads, D, G, None)


@pytest.mark.parametrize("fn", ["wq_kv_write", "wq_kv_read"])
def test_rows_refusals(L, fn):
    assert rows_call(L, fn, rows=0, batch=0) == 0              # nothing to do
    assert rows_call(L, fn, D=80, G=80) == 2
    assert rows_call(L, fn, G=48) == 1
    assert rows_call(L, fn, G=16) == 2
    assert rows_call(L, fn, page=24) == 2
    assert rows_call(L, fn, page=8) == 2
    assert rows_call(L, fn, heads=0) == 1
    assert rows_call(L, fn, dt=2) == 1
    assert rows_call(L, fn, rows=-1) == 1
    assert rows_call(L, fn, rows=3) == 1                       # 3 rows of 2 sequences without offsets
    assert rows_call(L, fn, rows=2, batch=0) == 1
    assert rows_call(L, fn, k=None) == 1
    assert rows_call(L, fn, v=None) == 1
    assert rows_call(L, fn, cache=None) == 1
    assert rows_call(L, fn, lens=None) == 1
    assert rows_call(L, fn, table=None) == 1
    assert rows_call(L, fn, k=136) == 2                        # misaligned
    assert rows_call(L, fn, cache=192) == 2
    assert rows_call(L, fn, ld_k=516) == 2                     # rows not 16-byte aligned
    assert rows_call(L, fn, ld_v=504) == 1                     # shorter than a row
    assert rows_call(L, fn, max_pages=1 << 27) == 2            # positions past 2^30
    assert rows_call(L, fn, rows=1 << 25, batch=1) == 2


def attend_call(L, q=128, ld_q=1024, dt=0, cache=128, table=4, lens=4, cu=None, out=128, ld_out=1024, rows=2, batch=2,
                max_pages=1, num_pages=4, page=16, q_heads=8, heads=4, D=128, G=128, scale=0.1, causal=1, window=0,
                max_kv=16, ws=None, ws_bytes=0):
    return L.wq_kv_attention(P(q), ld_q, dt, P(cache), P(table), P(lens), P(cu), P(out), ld_out, rows, batch, max_pages,
                             num_pages, page, q_heads, heads, D, G, scale, causal, window, max_kv, P(ws), ws_bytes, None)


def test_attention_refusals(L):
    assert attend_call(L, rows=0, batch=0) == 0
    assert attend_call(L, q_heads=6) == 1                      # not a multiple of the kv heads
    assert attend_call(L, q_heads=0) == 1
    assert attend_call(L, q_heads=8192) == 2
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert attend_call(L, scale=scale) == 1
    assert attend_call(L, causal=2) == 1
    assert attend_call(L, window=-1) == 1
    assert attend_call(L, max_kv=-1) == 1
    assert attend_call(L, dt=3) == 1
    assert attend_call(L, D=160, G=32) == 2
    assert attend_call(L, out=None) == 1
    assert attend_call(L, out=136) == 2
    assert attend_call(L, ld_q=1028) == 2
    assert attend_call(L, ld_out=512) == 1
    assert attend_call(L, rows=1 << 24, batch=1, q_heads=128, ld_q=1 << 20, ld_out=1 << 20, max_kv=0) == 2
    need = L.wq_kv_workspace_bytes(2, 2, 0, 8, 4, 128, 128, 100000)
    assert need > 0
    assert attend_call(L, max_kv=100000) == 4                  # workspace missing, short, misaligned
    assert attend_call(L, max_kv=100000, ws=128, ws_bytes=need - 1) == 4
    assert attend_call(L, max_kv=100000, ws=136, ws_bytes=need) == 2


def test_workspace_bytes(L):
    assert wq.wq_kv_workspace_bytes(1, 1, False, 32, 32, 128, 128, 64) == 0         # one part
    assert wq.wq_kv_workspace_bytes(4096, 64, False, 64, 8, 128, 128, 100000) == 0  # enough workgroups
    for bad in ((0, 1, 32, 32, 128), (3, 2, 32, 32, 128), (1, 1, 33, 32, 128), (1, 1, 32, 32, 96)):
        assert wq.wq_kv_workspace_bytes(bad[0], bad[1], False, bad[2], bad[3], bad[4], 64, 100000) == 0
    # parts x rows x heads x (sums, reference, weight)
    one = wq.wq_kv_workspace_bytes(1, 1, False, 8, 8, 128, 64, 1 << 20)
    assert one % (8 * (128 + 2) * 4) == 0 and 2 <= one // (8 * (128 + 2) * 4) <= 128


def meets(a, ld_a, b, ld_b, rows, width):
    """Whether two row matrices share an element, by counting (addresses in bytes)."""
    e = {a // 2 + i * ld_a + j for i in range(rows) for j in range(width)}
    return any(b // 2 + i * ld_b + j in e for i in range(rows) for j in range(width))


def test_shared_rows_are_refused(L):
    """Outputs over other rows' inputs, or over each other, are refused, slices that lie between each other's rows are
    not.  (Pointers are never read: what is not refused for its overlap ends at the missing workspace.)"""
    base, width = 1 << 20, 8 * 64
    for rows, ld_q, ld_out in ((2, 512, 512), (2, 1536, 1536), (4, 1024, 1024), (3, 1536, 1024), (3, 520, 1032), (1, 512, 512)):
        for d in sorted({i * 8 + o for i in (-3 * 192, -2 * 192, -192, -129, -128, -65, -64, -63, 0, 63, 64, 65, 128, 192)
                         for o in (-8, 0, 8)}):
            out = base + 2 * d
            shared = meets(base, ld_q, out, ld_out, rows, width) and not (d == 0 and (rows == 1 or ld_q == ld_out))
            assert attend_call(L, q=base, ld_q=ld_q, out=out, ld_out=ld_out, rows=rows, batch=rows, D=64, G=64, q_heads=8,
                               max_kv=100000) == (1 if shared else 4), (rows, ld_q, ld_out, d)
    # a long matrix with rows between the other's, strides that differ, and strides no memory has
    assert attend_call(L, q=base, out=base + 2 * 512 * 5, ld_q=1024, ld_out=512, rows=1 << 14, batch=1 << 14, D=64, G=64,
                       q_heads=8) == 1
    assert attend_call(L, q=base, out=base + 16, ld_q=1 << 62, ld_out=1 << 61, D=64, G=64, q_heads=8) == 1
    assert attend_call(L, q=base, out=base + 1024, ld_q=1 << 62, ld_out=1 << 61, D=64, G=64, q_heads=8, max_kv=100000) == 4
    # keys and values read back over each other
    for v, ld_k, ld_v in ((base, 512, 512), (base + 2 * 504, 512, 512), (base - 2 * 504, 512, 512), (base + 2 * 512, 512, 512),
                          (base + 2 * 520, 1024, 1024), (base + 1024, 1024, 512)):
        assert rows_call(L, "wq_kv_read", k=base, v=v, ld_k=ld_k, ld_v=ld_v) == 1, (v, ld_k, ld_v)


def test_workspace_of_lengths_past_32_bits(L):
    """The size asked for is the size the call asks of its workspace, whatever length is expected."""
    args = (1, 1, False, 8, 8, 128, 128)
    most = wq.wq_kv_workspace_bytes(*args, 1 << 30)
    assert most > wq.wq_kv_workspace_bytes(*args, 5000) > 0
    for n in ((1 << 30) + 1, 1 << 31, (1 << 32) + 5000, 1 << 40):
        assert wq.wq_kv_workspace_bytes(*args, n) == most, n


@pytest.fixture(scope="module")
def cache(L):
    return wq.wq_kv_cache(4, 16, 2, 64, 64, torch.float16, device="cpu")


def seqs(batch=2, pages=2):
    return torch.zeros(batch, pages, dtype=torch.int32), torch.ones(batch, dtype=torch.int32)


def rows_of(n=2, heads=2, D=64, dtype=torch.float16):
    return torch.zeros(n, heads, D, dtype=dtype)


def test_binding_refuses(cache):
    t, l = seqs()
    x = rows_of()
    with pytest.raises(wq.WQError):
        wq.wq_kv_cache(4, 16, 2, 80, 16, torch.float16, device="cpu")
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        wq.wq_kv_cache(4, 16, 2, 64, 64, torch.float32, device="cpu")
    for k, match in ((rows_of(dtype=torch.bfloat16), "cache's dtype"), (rows_of(heads=3), "2 heads"),
                     (rows_of(D=128), "head_dim 64"), (rows_of()[:, :, None], "heads..head_dim"),
                     (torch.zeros(2, 64, 2, dtype=torch.float16).transpose(1, 2), "contiguous"),
                     (torch.zeros(2, 132, dtype=torch.float16)[:, :128].view(2, 2, 64), "multiple of 8"),
                     (torch.zeros(300, dtype=torch.float16)[1:257].view(2, 2, 64), "16-byte aligned"),
                     (torch.zeros(1, 2, 64, dtype=torch.float16).expand(2, 2, 64), "row stride")):
        with pytest.raises(ValueError, match=match):
            wq.wq_kv_write(k, x, cache, t, l)
    with pytest.raises(ValueError, match="v must have 2 rows"):
        wq.wq_kv_write(x, rows_of(3), cache, t, l)
    with pytest.raises(ValueError, match="block_table"):
        wq.wq_kv_write(x, x, cache, t.long(), l)
    with pytest.raises(ValueError, match="block_table"):
        wq.wq_kv_write(x, x, cache, torch.zeros(2, 4, dtype=torch.int32)[:, ::2], l)
    with pytest.raises(ValueError, match="kv_lens"):
        wq.wq_kv_write(x, x, cache, t, l[:1])
    with pytest.raises(ValueError, match="cu_q"):
        wq.wq_kv_read(cache, t, l, 2, cu_q=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="as many rows"):
        wq.wq_kv_read(cache, t, l, 3)
    with pytest.raises(ValueError, match="out.1."):
        wq.wq_kv_read(cache, t, l, 2, out=(x, rows_of(3)))
    with pytest.raises(ValueError, match="multiple of the cache's 2 heads"):
        wq.wq_kv_attention(rows_of(heads=3), cache, t, l)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ValueError, match="scale"):
            wq.wq_kv_attention(x, cache, t, l, scale=scale)
    with pytest.raises(ValueError, match="window"):
        wq.wq_kv_attention(x, cache, t, l, window=-5)
    with pytest.raises(ValueError, match="out must have 2 rows"):
        wq.wq_kv_attention(x, cache, t, l, out=rows_of(3))
    with pytest.raises(ValueError, match="ws holds fewer"):
        wq.wq_kv_attention(x, cache, t, l, max_kv_len=100000, ws=torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="num_pages"):
        wq.KVCache(cache.data, (1 << 32) + 4, 16, 2, 64, 64, torch.float16)
    short = wq.KVCache(cache.data[:-1], 4, 16, 2, 64, 64, torch.float16)
    with pytest.raises(ValueError, match="shorter"):
        wq.wq_kv_write(x, x, short, t, l)
    for call in (lambda: wq.wq_kv_write(x, x, cache, t, l), lambda: wq.wq_kv_read(cache, t, l, 2),
                 lambda: wq.wq_kv_attention(x, cache, t, l)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_reference_codes(dt):
    """The reference's codes are the rationally nearest ones (the upper one half way)."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(6, 1, 32, generator=g).to(dt)
    x[0, 0] = torch.linspace(-1, 1, 32).to(dt)
    x[1, 0, ::2] = 0
    c, s, lo = _kv.quantise(x, 32)
    for t in range(6):
        step, base = fractions.Fraction(float(s[t, 0, 0])), fractions.Fraction(float(lo[t, 0, 0]))
        for e in range(32):
            d = fractions.Fraction(torch.tensor(float(x[t, 0, e]) - float(base), dtype=torch.float32).item())
            want = min(15, max(0, (d / step + fractions.Fraction(1, 2)).__floor__()))
            assert int(c[t, 0, 0, e]) == want


def test_reference_attention_is_softmax():
    P_ = _kv.Problem([7], [3], 1, 64, 64, 16, torch.float16, 1)
    q = P_.queries(2)
    out, bound = P_.reference(q, 0.2)
    K, V = (_kv.values(*_kv.quantise(x, 64))[:, 0] for x in (P_.K[0], P_.V[0]))
    for i in range(3):
        a = torch.softmax(q[i].double() @ K[:5 + i].T * 0.2, 1) @ V[:5 + i]
        assert torch.allclose(a, out[i], atol=1e-12)
    assert float(bound.max()) < 0.02


# ---------------------------------------------------------------------------
# Epilogue products
# ---------------------------------------------------------------------------
def epilogue_call(L, fn, bias=16, act=0, res=16, y=1 << 20, M=1, N=4096, K=4096, x=16):
    return getattr(L, fn)(P(x), 0, P(16), 0, None, None, P(bias), act, P(res), P(y), M, N, K, 4, 128, None, 0, None)


@pytest.mark.parametrize("fn", ["wq_gemv_epilogue", "wq_gemm_epilogue"])
def test_epilogue_refusals(L, fn):
    assert epilogue_call(L, fn, M=0) == 0
    assert epilogue_call(L, fn, act=4) == 1
    assert epilogue_call(L, fn, act=-1) == 1
    assert epilogue_call(L, fn, bias=24) == 2                      # misaligned
    assert epilogue_call(L, fn, res=24) == 2
    assert epilogue_call(L, fn, res=(1 << 20) + 16) == 1           # overlaps y without being y
    assert epilogue_call(L, fn, res=(1 << 20) - 16) == 1
    assert epilogue_call(L, fn, x=1 << 20) == 1                     # the layer's input as its output
    assert epilogue_call(L, fn, x=1 << 20, res=1 << 20) == 1        # x += layer(x)
    assert epilogue_call(L, fn, x=(1 << 20) - 8176) == 1            # x ends 16 bytes into y
    assert epilogue_call(L, fn, bias=(1 << 20) + 8176) == 1         # bias begins 16 bytes before y's end
    assert epilogue_call(L, fn, x=None) == 1
    assert epilogue_call(L, fn, N=4104) == 2
    assert epilogue_call(L, "wq_gemv_epilogue", M=33) == 2


def test_epilogue_binding_refuses(L):
    nbytes = wq.wq_packed_bytes(256, 64, 4, 128, wq.SYM)
    layer = wq.PackedLayer(torch.zeros(nbytes, dtype=torch.uint8), 256, 64, 4, 128, wq.SYM)
    x = torch.zeros(2, 256, dtype=torch.float16)
    half = dict(dtype=torch.float16)
    with pytest.raises(ValueError, match="act must be"):
        wq.linear(x, layer, act="tanh")
    with pytest.raises(ValueError, match="bias must have shape"):
        wq.linear(x, layer, bias=torch.zeros(63, **half))
    with pytest.raises(ValueError, match="bias must have dtype"):
        wq.linear(x, layer, bias=torch.zeros(64))
    with pytest.raises(ValueError, match="residual must have shape"):
        wq.linear(x, layer, residual=torch.zeros(1, 64, **half))
    with pytest.raises(ValueError, match="residual must be contiguous"):
        wq.wq_gemm_epilogue(x, layer, residual=torch.zeros(64, 2, **half).t())
    fused = wq.PackedLayer(layer.packed, 256, 64, 4, 128, wq.SYM, gate_up=True)
    with pytest.raises(ValueError, match="wq_repack"):
        wq.linear(x, fused, bias=torch.zeros(64, **half))
    with pytest.raises(ValueError, match="GPU tensor"):
        wq.linear(x, layer, bias=torch.zeros(64, **half))
