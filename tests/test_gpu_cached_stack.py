"""Decoder layers with attention over the 4-bit cache (weight_only_quantized_w4a16_amd.stack.CachedStack).

Every part is checked on the very input the GPU used: products against the
oracle (with bias and residual in 64 bits), attention against the 64-bit
reference on the keys and values the products gave.  A prompt in one step, in
ragged chunks and token by token go through the same layers; a decode step is
captured once and replayed as the sequences grow."""
import numpy as np
import pytest
import torch

import _kv
import workloads as wl
from _util import bits_to_tensor, oracle_y, repack_layer, tensor_bits, tensor_f64, within_tolerance
from test_gpu_gate_up import gate_up_bound, repack_gate_up

pytestmark = pytest.mark.gpu
DIM, INTER, H, KV, D = 512, 768, 8, 2, 64
QKV = (H + 2 * KV) * D


@pytest.fixture(scope="module")
def wq():
    import weight_only_quantized_w4a16_amd as m
    m.lib()
    assert torch.cuda.is_available()
    return m


@pytest.fixture(scope="module")
def weights(wq):
    from weight_only_quantized_w4a16_amd.stack import DecoderWeights
    layers, raw = [], []
    for li in range(2):
        Ls = {}
        for j, (name, K, N) in enumerate((("qkv", DIM, QKV), ("o", H * D, DIM), ("gate_up", DIM, 2 * INTER),
                                          ("down", INTER, DIM))):
            c = 0.5 / np.sqrt(13.0 / 12.0 * 22.6 * K)
            Ls[name] = wl.make_layer(K, N, 4, 128, wl.ZERO_F16, 100 * li + j, scale_range=(0.5 * c, 1.5 * c),
                                     zero_range=(5.5, 9.5))
        layers.append(DecoderWeights(repack_layer(wq, Ls["qkv"]), repack_layer(wq, Ls["o"]),
                                     repack_gate_up(wq, Ls["gate_up"]), repack_layer(wq, Ls["down"])))
        raw.append(Ls)
    g = torch.Generator().manual_seed(4)
    bias = [(torch.randn(QKV, generator=g) * 0.3).half().cuda() for _ in layers]
    return layers, raw, bias


def make_stack(weights, max_rows, pages=40):
    from weight_only_quantized_w4a16_amd.stack import CachedStack
    layers, _, bias = weights
    return CachedStack(layers, H, KV, D, pages, max_rows, torch.float16, "cuda", qkv_bias=bias)


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def add_ok(orc, x, L, y, plus):
    """y = x W + plus within the products' tolerance of the 64-bit sum."""
    ref = oracle_y(orc, tensor_bits(x), wl.F16, L)
    _, _, bound = within_tolerance(ref, ref)
    want = ref + plus
    err = float(np.max(np.abs(tensor_f64(y) - want)))
    assert err <= bound + 2.0 ** -11 * float(np.max(np.abs(want))), (err, bound)


def check_step(orc, rec, raw, bias, hist, new, lens):
    """hist[layer][sequence]: K and V rows so far (on the CPU), extended by this step's."""
    for r, Ls, b in zip(rec, raw, bias):
        T = r["x"].shape[0]
        add_ok(orc, r["x"], Ls["qkv"], r["qkv"], tensor_f64(b))
        heads = r["qkv"].view(T, H + 2 * KV, D).cpu()
        at = 0
        for s, n in enumerate(new):
            rows = heads[at:at + n]
            K, V = hist[r["layer"]][s]
            K, V = torch.cat([K, rows[:, H:H + KV]]), torch.cat([V, rows[:, H + KV:]])
            hist[r["layer"]][s] = (K, V)
            assert K.shape[0] == lens[s]
            want, bound = _kv.attention(rows[:, :H], K, V, torch.arange(lens[s] - n, lens[s]), D ** -0.5, True, 0, D)
            assert bool(((r["attn"][at:at + n].cpu().double() - want).abs() <= bound).all())
            at += n
        add_ok(orc, r["attn"].reshape(T, H * D), Ls["o"], r["mid"], tensor_f64(r["x"]))
        L = Ls["gate_up"]
        mb = tensor_bits(r["mid"])
        h_ref = orc.linear_gate_up(mb, wl.F16, L.qweight, L.scales, L.zeros, L.mode, L.lut, L.g_idx, T, L.N, L.K,
                                   L.bits, L.group_size)
        assert np.all(np.abs(tensor_f64(r["h"]) - h_ref) <= gate_up_bound(oracle_y(orc, mb, wl.F16, L), h_ref, wl.F16))
        add_ok(orc, r["h"], Ls["down"], r["y"], tensor_f64(r["mid"]))


def empty_history(n):
    e = torch.empty(0, KV, D, dtype=torch.float16)
    return [[(e, e) for _ in range(n)] for _ in range(2)]


def test_prompt_chunks_and_tokens(orc, wq, weights):
    _, raw, bias = weights
    st = make_stack(weights, 80)
    table = i32([[3, 9, 1, 30, 31], [17, 0, 2, 22, 5], [11, 12, 13, 14, 15]])
    hist = empty_history(3)
    lens = [0, 0, 0]
    g = torch.Generator().manual_seed(9)
    # prompts, a chunk behind some of them beside a new prompt, then single tokens
    for new in ([45, 3, 0], [1, 20, 33], [1, 1, 1], [1, 1, 1]):
        lens = [a + b for a, b in zip(lens, new)]
        x = torch.randn(sum(new), DIM, generator=g).half().cuda()
        cu = None if len(set(new)) == 1 else i32([0] + list(np.cumsum(new)))
        rec = []
        y = st.step(x, table, i32(lens), cu, max_kv_len=max(lens), record=rec)
        assert torch.equal(rec[-1]["y"], y) and torch.equal(rec[1]["x"], rec[0]["y"])
        check_step(orc, rec, raw, bias, hist, new, lens)


def test_one_prompt_in_any_pieces(wq, weights):
    """The cache holds the same codes however a prompt was cut, and the outputs agree to the products' tolerance."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(50, DIM, generator=g).half().cuda()
    table = i32([[0, 1, 2, 3]])
    whole = make_stack(weights, 50).step(x, table, i32([50])).clone()
    st = make_stack(weights, 50)
    parts, at = [], 0
    for n in (17, 1, 1, 31):
        parts.append(st.step(x[at:at + n].contiguous(), table, i32([at + n])).clone())
        at += n
    got = torch.cat(parts)
    # each of the four products and the attention may round differently: 2 layers x 5 parts, each within the products tolerance
    assert float((got - whole).abs().max()) <= 10 * (5e-3 * float(whole.abs().max()) + 1e-3)


def test_decode_step_in_a_graph(wq, weights):
    g = torch.Generator().manual_seed(3)
    prompt = torch.randn(2 * 30, DIM, generator=g).half().cuda()
    table = i32([[0, 1, 2, 3], [4, 5, 6, 7]])
    tokens = [torch.randn(2, DIM, generator=g).half().cuda() for _ in range(4)]
    eager, st = make_stack(weights, 60), make_stack(weights, 60)
    for s in (eager, st):
        s.step(prompt, table, i32([30, 30]))
    want = [eager.step(t, table, i32([31 + i, 31 + i]), max_kv_len=64).clone() for i, t in enumerate(tokens)]
    x, lens = tokens[0].clone(), i32([31, 31])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = st.step(x, table, lens, max_kv_len=64)
    for i, t in enumerate(tokens):
        x.copy_(t)
        lens.fill_(31 + i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), i


def test_step_on_another_stream(wq, weights):
    """Scratch allocated for a step on a side stream is not handed out under it."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(40, DIM, generator=g).half().cuda()
    table = i32([[0, 1, 2, 3]])
    want = make_stack(weights, 40).step(x, table, i32([40]), max_kv_len=100000).clone()
    st = make_stack(weights, 40)
    side = torch.cuda.Stream()
    lens = i32([40])
    torch.cuda.synchronize()
    out = st.step(x, table, lens, max_kv_len=100000, stream=side)
    junk = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(32)]
    side.synchronize()
    assert torch.equal(out, want) and len(junk) == 32


def test_stack_refusals(wq, weights):
    from weight_only_quantized_w4a16_amd.stack import CachedStack
    layers, _, bias = weights
    with pytest.raises(ValueError, match="chain"):
        CachedStack(layers, H, 4, D, 8, 4, torch.float16, "cuda")
    with pytest.raises(ValueError, match="bias"):
        CachedStack(layers, H, KV, D, 8, 4, torch.float16, "cuda", qkv_bias=bias[:1])
    st = make_stack(weights, 2)
    with pytest.raises(ValueError, match="max_rows"):
        st.step(torch.zeros(3, DIM, dtype=torch.float16, device="cuda"), i32([[0]]), i32([3]))


def test_record_on_another_stream(wq, weights):
    """The recorded tensors are copied where the work is: a step given to a busy stream records what it computes, and
    its input also where the layer writes its output over it."""
    from weight_only_quantized_w4a16_amd.stack import CachedStack, DecodeStack, DecoderWeights
    layers, raw, bias = weights
    g = torch.Generator().manual_seed(6)
    x = torch.randn(3, DIM, generator=g).half().cuda()
    table, lens = i32([[0], [1], [2]]), i32([1, 1, 1])
    # (the chain without a cache takes the first columns of its QKV output into a projection of DIM columns)
    plain = [DecoderWeights(layers[0].qkv, layers[0].o, layers[0].gate_up, layers[0].down)]
    cached = CachedStack(layers[:1], H, KV, D, 8, 3, torch.float16, "cuda", qkv_bias=bias[:1])
    side = torch.cuda.Stream()
    a = torch.randn(4096, 4096, device="cuda").half()
    b = torch.empty_like(a)
    for st, args in ((cached, (table, lens)), (DecodeStack(plain, 3, torch.float16, "cuda"), ())):
        want = []
        y = st.step(x, *args, record=want).clone()
        again = []
        st.step(st.step(x, *args), *args, record=again)  # its own output buffer as the input
        torch.cuda.synchronize()
        assert torch.equal(again[0]["x"], y)
        assert torch.equal(want[0]["y"], y) and torch.equal(want[0]["x"], x)
        for t in vars(st).values():
            for buf in t if isinstance(t, list) else [t]:
                if isinstance(buf, torch.Tensor) and buf.dtype == torch.float16 and buf.is_cuda and buf.shape[-1] != QKV:
                    buf.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(40):
                torch.mm(a, a, out=b)
        rec = []
        st.step(x, *args, stream=side, record=rec)
        side.synchronize()
        assert rec[0].keys() == want[0].keys() and rec[0]["layer"] == 0
        for name, t in want[0].items():
            assert name == "layer" or torch.equal(rec[0][name], t), name
